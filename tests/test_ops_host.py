"""The operators' host side on the CPU: argument checks of the stateless calls
(made before any device work), the compaction plan, and the page calls of a
handle under AddressSanitizer and UndefinedBehaviorSanitizer with a device
double, refusals and bookkeeping included."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ric():
    from ragged_input_compilation_amd import _ric
    return _ric


def code(ric, fn, *a, **kw):
    with pytest.raises(ric.RicError) as e:
        fn(*a, **kw)
    return e.value.code


def _attention(ric, **kw):
    base = dict(dtype=ric.RIC_BF16, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16, scale=0.1, softcap=0.0,
                window=0, alibi_slopes=0, prefix_lens=0)
    return ric.make_attention(**{**base, **kw})


# Addresses that no call may follow: every case below is refused, or has nothing to do.
CALL = dict(q=4096, k_cache=4096, v_cache=4096, num_blocks=10, block_table=4096, block_table_stride=4,
            block_table_width=4, query_start_loc=4096, seq_lens=4096, num_reqs=2, num_tokens=2, max_query_len=1,
            max_seq_len=20, out=4096)


def test_attention_refusals(ric):
    for kw in (dict(dtype=ric.RIC_F32), dict(dtype=7), dict(num_heads=0), dict(num_kv_heads=0), dict(num_heads=9),
               dict(num_heads=70000, num_kv_heads=70000), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264),
               dict(block_size=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0),
               dict(softcap=float("nan")), dict(softcap=float("inf")), dict(window=-1), dict(window=(1 << 30) + 1),
               dict(num_heads=520, num_kv_heads=4)):
        a = _attention(ric, **kw)
        assert code(ric, ric.ric_paged_attention, a, **CALL) == ric.RIC_EINVAL, kw
        assert ric.ric_paged_attention_workspace_bytes(a, 2, 2, 1, 20) == 0
    a = _attention(ric)
    for kw in (dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(block_table=0), dict(query_start_loc=0),
               dict(seq_lens=0), dict(out=0), dict(q=4104), dict(k_cache=4100), dict(v_cache=4098), dict(out=4097),
               dict(q_stride=2040), dict(q_stride=2056), dict(out_stride=16), dict(num_blocks=0),
               dict(num_blocks=1 << 27), dict(num_blocks=1 << 40), dict(block_table_width=5), dict(block_table_width=-1),
               dict(num_reqs=-1), dict(num_tokens=-1), dict(num_tokens=(1 << 22) + 1), dict(num_reqs=(1 << 22) + 1),
               dict(max_query_len=-1), dict(max_seq_len=-1)):
        assert code(ric, ric.ric_paged_attention, a, **{**CALL, **kw}) == ric.RIC_EINVAL, kw
    ric.ric_paged_attention(a, **{**CALL, "num_reqs": 0})          # nothing to do
    ric.ric_paged_attention(a, **{**CALL, "num_tokens": 0, "q": 0, "out": 0})
    # long axes take a workspace, which is checked
    need = ric.ric_paged_attention_workspace_bytes(a, 1, 1, 1, 100000)
    if need:
        long = {**CALL, "num_reqs": 1, "num_tokens": 1, "max_seq_len": 100000}
        for ws in (dict(), dict(workspace=4096, workspace_bytes=need - 256 - 1), dict(workspace=4104, workspace_bytes=need)):
            assert code(ric, ric.ric_paged_attention, a, **{**long, **ws}) == ric.RIC_EINVAL, ws


def test_attention_workspace_does_not_depend_on_the_mask(ric):
    """One workspace serves the layers of a model with and without windows."""
    rng = np.random.default_rng(1)
    for _ in range(400):
        reqs, q = int(rng.integers(1, 300)), int(rng.integers(1, 70))
        kv = int(rng.choice([1, 2, 8]))
        args = (reqs, reqs * q, q, int(np.exp(rng.uniform(0, 13))))
        kw = dict(num_kv_heads=kv, num_heads=kv * int(rng.choice([1, 4, 8])), head_dim=int(rng.choice([64, 128, 80])))
        base = ric.ric_paged_attention_workspace_bytes(_attention(ric, **kw), *args)
        for w in (1, 500, 1024, 5000, 32768, 1 << 30):
            assert ric.ric_paged_attention_workspace_bytes(_attention(ric, window=w, **kw), *args) == base
        assert base < 1 << 30


def test_logprobs_refusals(ric):
    ok = dict(logits=4096, dtype=ric.RIC_BF16, targets=4096, max_rows=3, vocab=100, top_k=5, logprob=4096, rank=4096,
              entropy=4096, top_ids=4096, top_logprobs=4096)
    for kw in (dict(dtype=3), dict(dtype=-1), dict(logits=0), dict(logits=4097), dict(dtype=ric.RIC_F32, logits=4098),
               dict(row_stride=198), dict(row_stride=201), dict(dtype=ric.RIC_F32, row_stride=402), dict(max_rows=-1),
               dict(max_rows=(1 << 22) + 1), dict(vocab=0), dict(vocab=-4), dict(top_k=-1), dict(top_k=65),
               dict(vocab=4), dict(targets=0), dict(logprob=0), dict(rank=0), dict(top_ids=0), dict(top_logprobs=0),
               dict(top_k=0)):
        assert code(ric, ric.ric_token_logprobs, **{**ok, **kw}) == ric.RIC_EINVAL, kw
    ric.ric_token_logprobs(**{**ok, "max_rows": 0})
    need = ric.ric_token_logprobs_workspace_bytes(1, 150000, 5)
    if need:
        for ws in (dict(), dict(workspace=4096, workspace_bytes=16), dict(workspace=4104, workspace_bytes=need)):
            assert code(ric, ric.ric_token_logprobs, **{**ok, "max_rows": 1, "vocab": 150000, **ws}) == ric.RIC_EINVAL


def test_logprobs_sizes(ric):
    """A workspace of a row count is enough for every smaller one."""
    for vocab, k in ((8192, 5), (16384, 0), (60001, 3), (151936, 64), (1 << 30, 64)):
        last = 0
        for rows in (1, 2, 3, 31, 32, 33, 100, 511, 512, 513, 1000, 1023, 1024, 5000, 1 << 22):
            need = ric.ric_token_logprobs_workspace_bytes(rows, vocab, k)
            pieces = max(1, min(-(-1024 // rows), vocab // 8192, 32))
            assert need >= max(last, 0 if pieces == 1 else rows * pieces * (16 + 8 * k))
            last = need
        assert last < 4 << 20
    assert ric.ric_token_logprobs_workspace_bytes(1, (1 << 30) + 1, 5) == 0
    assert code(ric, ric.ric_token_logprobs, logits=4096, dtype=ric.RIC_BF16, targets=0, max_rows=1,
                vocab=(1 << 30) + 1, top_k=0, logprob=0, rank=0, entropy=0, top_ids=0, top_logprobs=0) == ric.RIC_EINVAL


def test_tensors_that_overlap_themselves_are_refused():
    """Expanded and overlapping rows have no stride the calls could take."""
    import torch
    from ragged_input_compilation_amd import runner
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    q, cache, table, qsl, seq = bf(2, 4, 64), bf(5, 16, 2, 64), i32(2, 3), i32(3), i32(2)
    call = lambda q=q, table=table, out=None: runner.paged_attention(q, cache, cache, table, qsl, seq, 1, 40,
                                                                     bf(2, 4, 64) if out is None else out)
    for kw in (dict(q=bf(1, 4, 64).expand(2, 4, 64)), dict(out=bf(1, 4, 64).expand(2, 4, 64)),
               dict(q=bf(600).as_strided((2, 4, 64), (128, 64, 1))), dict(table=i32(1, 3).expand(2, 3)),
               dict(table=i32(9).as_strided((2, 3), (2, 1)))):
        with pytest.raises(ValueError):
            call(**kw)
    for logits in (bf(1, 100).expand(4, 100), bf(400).as_strided((4, 100), (50, 1))):
        with pytest.raises(ValueError):
            runner.token_logprobs(logits, None, 0)


def test_compact_plan(ric):
    rng = np.random.default_rng(0)
    for _ in range(300):
        n = int(rng.integers(1, 60))
        null = int(rng.integers(0, n))
        refs = (rng.random(n) < rng.random()).astype(np.int32) * rng.integers(1, 4, n).astype(np.int32)
        src, dst = ric.ric_compact_plan(refs, null)
        after = refs.copy()
        for s, d in zip(src, dst):
            assert refs[s] > 0 and refs[d] <= 0 and d < s and null not in (s, d)
            after[d], after[s] = after[s], 0
        used = [i for i in range(n) if after[i] > 0 and i != null]
        assert used == [i for i in range(n) if i != null][:len(used)]
        assert list(dst) == sorted(dst) and list(src) == sorted(src, reverse=True)
    assert [len(x) for x in ric.ric_compact_plan([])] == [0, 0]


_CHILD = r"""
import ctypes, sys
import numpy as np
sys.path.insert(0, {root!r})
from ragged_input_compilation_amd import _ric as ric

def words(ptr, n):
    return np.ctypeslib.as_array((ctypes.c_int32 * max(n, 1)).from_address(ptr))[:n].copy()

def rejects(fn, *a, **kw):
    try:
        fn(*a, **kw)
    except ric.RicError as e:
        return e.code
    raise AssertionError("accepted")

B, POOL, ROW, MB = 4, 9000, 16, 12
cfg = ric.make_config(max_num_reqs=8, max_model_len=48, block_size=B, max_blocks_per_req=MB, max_num_batched_tokens=64,
                      num_kv_blocks=POOL, null_block=0, staging_bytes=2 * 12 * 8 * 4 + (64 << 10))
h = ric.ric_create(cfg, 0)
rng = np.random.default_rng(3)
kc = [rng.integers(0, 256, (POOL, B * ROW)).astype(np.uint8) for _ in range(2)]
vc = [rng.integers(0, 256, (POOL, B * ROW)).astype(np.uint8) for _ in range(2)]
raw = []
def aligned(a):
    buf = np.zeros(a.nbytes + 16, np.uint8)
    off = -buf.ctypes.data % 16
    v = buf[off:off + a.nbytes].reshape(a.shape)
    v[:] = a
    raw.append(buf)
    return v
kc, vc = [aligned(x) for x in kc], [aligned(x) for x in vc]
kp, vp = [x.ctypes.data for x in kc], [x.ctypes.data for x in vc]
tables = {{}}
toks = {{}}
free = list(rng.permutation(np.arange(1, POOL)))
for i in range(3):
    toks[i] = rng.integers(0, 99, 20).tolist()
    tables[i] = [int(free.pop()) for _ in range(6)]
    ric.ric_add_request(h, i, toks[i], 10, 0, tables[i], (0.5, 0.6, 0.7, i))

def check():
    ric.ric_flush(h)
    cols = ric.ric_get_columns(h)
    for i in tables:
        r = ric.ric_row_of(h, i)
        assert list(words(cols.blocks + 4 * r * cols.block_stride, len(tables[i]))) == tables[i], i
        assert list(words(cols.tokens + 4 * r * cols.token_stride, len(toks[i]))) == toks[i], i
        assert words(cols.num_blocks + 4 * r, 1)[0] == len(tables[i])
        assert words(cols.num_tokens + 4 * r, 1)[0] == len(toks[i])

# copies, more than one launch's pairs
n = 4300
ids = rng.permutation(np.asarray(free))[:2 * n]
want = [x.copy() for x in kc + vc]
for x in want:
    x[ids[n:]] = x[ids[:n]]
ric.ric_copy_blocks(h, ids[:n], ids[n:], kp, vp, B * ROW)
assert all(np.array_equal(a, b) for a, b in zip(kc + vc, want))
# moves: tables follow
src = [tables[0][1], tables[2][5], tables[1][0]]
dst = [int(free.pop()) for _ in range(3)]
want = [x.copy() for x in kc + vc]
for x in want:
    x[dst] = x[src]
ric.ric_schedule(h, [0, 0, 0], [1, 1, 1])
ric.ric_move_blocks(h, src, dst, kp, vp, B * ROW)
assert all(np.array_equal(a, b) for a, b in zip(kc + vc, want))
tables = {{i: [dict(zip(src, dst)).get(x, x) for x in t] for i, t in tables.items()}}
check()
assert rejects(ric.ric_compile, h, 8) == ric.RIC_ESTATE
refs = np.full(POOL, 5, np.int32)
ric.ric_block_refs(h, refs.ctypes.data)
assert np.array_equal(refs, np.bincount(sum(tables.values(), []), minlength=POOL))
# forks
for child, T, c, new in ((10, 20, 10, 2), (11, 15, 8, 1), (12, 10, 0, 0), (13, 20, 20, 0)):
    nb = [int(free.pop()) for _ in range(new)]
    tail = c % B
    want = [x.copy() for x in kc + vc]
    for x in want:
        if tail:
            x[nb[0], :tail * ROW] = x[tables[1][c // B], :tail * ROW]
    ric.ric_append_tokens(h, 1, [7])              # still staged when the fork reads the row
    toks[1] = toks[1] + [7]
    ric.ric_fork_request(h, 1, child, T, c, nb, kp, vp, ROW)
    toks[child] = toks[1][:T]
    tables[child] = tables[1][:c // B] + nb
    assert all(np.array_equal(a, b) for a, b in zip(kc + vc, want)), child
    check()
# refusals change nothing
f = lambda *a, **kw: rejects(ric.ric_fork_request, h, *a, **kw)
assert f(99, 30, 10, 0, []) == ric.RIC_ENOENT
assert f(1, 10, 10, 0, []) == ric.RIC_EEXIST
assert f(1, 30, 9, 0, []) == ric.RIC_ERANGE                       # below the prompt
assert f(1, 30, len(toks[1]) + 1, 0, []) == ric.RIC_ERANGE
assert f(1, 30, 12, 13, [5]) == ric.RIC_ERANGE
assert f(1, 30, 12, -1, [5]) == ric.RIC_ERANGE
assert f(1, 30, 12, 5, []) == ric.RIC_EINVAL                      # a partial page needs a block
assert f(1, 30, 12, 5, [0]) == ric.RIC_ERANGE                     # the null block
assert f(1, 30, 12, 5, [POOL]) == ric.RIC_ERANGE
assert f(1, 30, 12, 8, [5] * 11) == ric.RIC_ERANGE                # table capacity
assert f(12, 30, 10, 1, [5]) == ric.RIC_ERANGE                    # the parent has no page for it
assert f(1, 30, 12, 5, [5], kp, vp, 24) == ric.RIC_EINVAL
assert f(1, 30, 12, 5, [5], [kp[0] + 8], [vp[0]], ROW) == ric.RIC_EINVAL
assert f(1, 30, 12, 5, [5], [0], [vp[0]], ROW) == ric.RIC_EINVAL
ric.ric_fork_request(h, 1, 14, 12, 8, [int(free.pop())])
assert f(1, 30, 12, 8, []) == ric.RIC_EFULL
ric.ric_remove_request(h, 14)
g = lambda fn, *a: rejects(fn, h, *a)
for fn in (ric.ric_copy_blocks, ric.ric_move_blocks):
    assert g(fn, [1], [0], kp, vp, 64) == ric.RIC_ERANGE
    assert g(fn, [0], [1], kp, vp, 64) == ric.RIC_ERANGE
    assert g(fn, [POOL], [1], kp, vp, 64) == ric.RIC_ERANGE
    assert g(fn, [1], [-1], kp, vp, 64) == ric.RIC_ERANGE
    assert g(fn, [1, 2], [3, 3], kp, vp, 64) == ric.RIC_EINVAL
    assert g(fn, [1, 2], [2, 3], kp, vp, 64) == ric.RIC_EINVAL
    assert g(fn, [4], [4], kp, vp, 64) == ric.RIC_EINVAL
    assert g(fn, [1], [2], kp, vp, 40) == ric.RIC_EINVAL
    assert g(fn, [1], [2], kp, vp, 0) == ric.RIC_EINVAL
    assert g(fn, [1], [2], [kp[0] + 4], [vp[0]], 64) == ric.RIC_EINVAL
    assert g(fn, [1], [2], [0], [vp[0]], 64) == ric.RIC_EINVAL
    assert g(fn, [1], [2], kp, vp, 64, 1) == ric.RIC_EINVAL          # no such group
assert g(ric.ric_move_blocks, [1, 1], [2, 3], kp, vp, 64) == ric.RIC_EINVAL
assert g(ric.ric_block_refs, 0) == ric.RIC_EINVAL
ric.lib().fake_set_capturing(1)
assert g(ric.ric_copy_blocks, [1], [2], kp, vp, 64) == ric.RIC_ESTATE
assert g(ric.ric_fork_request, 1, 30, 12, 8, []) == ric.RIC_ESTATE
ric.lib().fake_set_capturing(0)
ric.ric_remove_request(h, 0)
assert g(ric.ric_move_blocks, [1], [2], kp, vp, 64) == ric.RIC_ESTATE      # a hole
assert g(ric.ric_block_refs, refs.ctypes.data) == ric.RIC_ESTATE
del tables[0], toks[0]
assert ric.ric_row_of(h, 30) == -1
check()
ric.ric_destroy(h)
print("page calls ok")
"""


def test_page_calls_under_asan_and_ubsan(tmp_path):
    asan = subprocess.run(["gcc", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("no AddressSanitizer runtime for gcc here")
    so = tmp_path / "libric_fake_ops.so"
    csrc = os.path.join(ROOT, "ragged_input_compilation_amd", "csrc")
    fake = os.path.join(ROOT, "tests", "host_fake")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    os.path.join(csrc, "ric_host.cpp"), os.path.join(csrc, "ric_ops_host.cpp"),
                    os.path.join(fake, "fake_device.cpp"), os.path.join(fake, "fake_ops.cpp"), "-o", str(so)], check=True)
    preload = ":".join(x for x in (asan, os.environ.get("LD_PRELOAD", "")) if x)   # ASan first, nothing removed
    env = {**os.environ, "LD_PRELOAD": preload, "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=1",
           "RIC_LIBRARY": str(so)}
    child = subprocess.run([sys.executable, "-c", _CHILD.format(root=ROOT)], capture_output=True, text=True,
                           timeout=600, env=env)
    assert child.returncode == 0, child.stdout[-2000:] + child.stderr[-4000:]
    assert "page calls ok" in child.stdout
    assert "AddressSanitizer" not in child.stderr and "runtime error" not in child.stderr
