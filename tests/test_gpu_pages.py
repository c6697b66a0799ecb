"""Pages copied, moved, counted and forked: every byte of every cache and every
live table entry against numpy, the steps that follow included."""
import numpy as np
import pytest
import torch

import workloads
from tests.gpu_helpers import read_rows_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ragged_input_compilation_amd import _ric, runner
    return _ric, runner


def make(rt, *, reqs=10, block=16, pool=400, groups=1, seed=0, max_len=256, max_reqs=None):
    ric, runner = rt
    rng = np.random.default_rng(seed)
    kw = {}
    if groups == 2:
        kw = dict(num_kv_groups=2, group_block_size=[0, 8], group_num_kv_blocks=[0, 300], group_slot_mode=[0, 0])
    b = runner.Batch(ric.make_config(max_num_reqs=max_reqs or reqs + 4, max_model_len=max_len, block_size=block,
                                     max_blocks_per_req=max_len // block, max_num_batched_tokens=1024,
                                     num_kv_blocks=pool, null_block=0, staging_bytes=0, **kw))
    ids = rng.permutation(np.arange(1, pool))
    ids1 = rng.permutation(np.arange(1, 300))
    tables, tables1, toks, at, at1 = [], [], [], 0, 0
    for i in range(reqs):
        T = int(rng.integers(1, max_len - 20))
        n = -(-T // block)
        toks.append(rng.integers(0, 1000, T).astype(np.int32))
        tables.append(ids[at:at + n].astype(np.int32))
        ric.ric_add_request(b.h, i, toks[i], max(1, T // 2), 0, tables[i], (0.5 + i, 0.9, 1.1, i))
        at += n
        if groups == 2:
            n1 = int(rng.integers(0, 12))
            tables1.append(ids1[at1:at1 + n1].astype(np.int32))
            ric.ric_append_blocks_group(b.h, i, 1, tables1[i])
            at1 += n1
    return b, tables, tables1, toks, rng


def caches(layers, pool, block, row, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [[torch.randint(0, 256, (pool, block, row), generator=g, device="cuda", dtype=torch.uint8)
             for _ in range(layers)] for _ in range(2)]


def expect(cs, src, dst):
    out = []
    for c in cs:
        w = c.clone()
        if len(src):
            w[torch.from_numpy(np.asarray(dst)).long().cuda()] = c[torch.from_numpy(np.asarray(src)).long().cuda()]
        out.append(w)
    return out


@pytest.mark.parametrize("layers,row,block,n", [(1, 16, 1, 1), (1, 48, 5, 7), (3, 256, 16, 30), (33, 64, 16, 12),
                                               (2, 2048, 16, 100), (1, 4096, 16, 9), (70, 16, 3, 4)])
def test_copy(rt, layers, row, block, n):
    ric, runner = rt
    pool = 250
    b, *_ , rng = make(rt, pool=pool, reqs=2, block=block, max_len=60)
    kc, vc = caches(layers, pool, block, row, n)
    ids = rng.permutation(np.arange(1, pool))
    dst = ids[:n]
    src = rng.choice(ids[n:], size=n)                       # a source may feed several destinations
    want_k, want_v = expect(kc, src, dst), expect(vc, src, dst)
    runner.copy_blocks(b, src, dst, kc, vc)
    for got, want in zip(kc + vc, want_k + want_v):
        assert torch.equal(got, want)
    runner.copy_blocks(b, [], [], kc, vc)
    for got, want in zip(kc + vc, want_k + want_v):
        assert torch.equal(got, want)
    b.close()


def test_more_pages_than_one_launch_holds(rt):
    ric, runner = rt
    pool = 12000
    b, *_, rng = make(rt, pool=pool, reqs=3)
    kc, vc = caches(2, pool, 16, 16, 5)
    ids = rng.permutation(np.arange(1, pool))
    src, dst = ids[:5500], ids[5500:11000]
    want_k, want_v = expect(kc, src, dst), expect(vc, src, dst)
    runner.copy_blocks(b, src, dst, kc, vc)
    for got, want in zip(kc + vc, want_k + want_v):
        assert torch.equal(got, want)
    b.close()


def test_pages_past_the_caches_are_refused(rt):
    ric, runner = rt
    b, *_ = make(rt, groups=2, pool=400, reqs=3)
    kc, vc = caches(2, 100, 16, 16, 5)
    for src, dst in (([1, 100], [2, 3]), ([1, 2], [3, 399])):
        for call in (runner.copy_blocks, runner.move_blocks):
            with pytest.raises(ValueError):
                call(b, src, dst, kc, vc)
    with pytest.raises(ValueError):
        runner.copy_blocks(b, [1], [2], kc, vc[:1])
    for group in (-1, 2):
        with pytest.raises(ValueError):
            runner.copy_blocks(b, [1], [2], kc, vc, group)
        with pytest.raises(ValueError):
            runner.block_refs(b, group)
    runner.copy_blocks(b, [1], [99], kc, vc)
    b.close()


@pytest.mark.parametrize("group", [0, 1])
def test_compaction_moves_pages_and_tables(rt, group):
    """refs -> plan -> move: the used pages become the lowest ones, every live
    entry follows, entries of the other group and stale ones do not."""
    ric, runner = rt
    b, t0, t1, _, rng = make(rt, groups=2, reqs=20, pool=400)
    for i in (3, 11, 19):
        ric.ric_remove_request(b.h, i)
    with pytest.raises(ric.RicError) as e:
        runner.block_refs(b, group)                         # rows are not condensed
    assert e.value.code == ric.RIC_ESTATE
    ric.ric_condense(b.h)
    order = b.row_order()
    tables = [list(map(int, (t0, t1)[group][i])) for i in order]
    others = [list(map(int, (t1, t0)[group][i])) for i in order]
    pool = (400, 300)[group]
    refs = runner.block_refs(b, group).cpu().numpy()
    want = np.bincount(np.concatenate([np.asarray(t, np.int64) for t in tables if len(t)]), minlength=pool)
    assert np.array_equal(refs, want)
    src, dst = ric.ric_compact_plan(refs)
    n_used = int((want > 0).sum())
    block = (16, 8)[group]
    kc, vc = caches(2, pool, block, 64, 9)
    before = [c.clone() for c in kc + vc]
    runner.move_blocks(b, src, dst, kc, vc, group)
    to = {int(s): int(d) for s, d in zip(src, dst)}
    cols = ric.ric_get_columns(b.h)
    for row, (mine, other) in enumerate(zip(tables, others)):
        for g, ids in ((group, [to.get(x, x) for x in mine]), (1 - group, other)):
            got = read_rows_i32(b.workspace, cols.group_blocks[g], cols.group_block_stride[g], [row], len(ids))[0]
            assert list(got) == ids
        for x in mine:                                       # the pages' bytes are where the tables say
            for c, old in zip(kc + vc, before):
                assert torch.equal(c[to.get(x, x)], old[x])
    refs = runner.block_refs(b, group).cpu().numpy()
    assert (refs[1:n_used + 1] > 0).all() and (refs[n_used + 1:] == 0).all()
    assert len(ric.ric_compact_plan(refs)[0]) == 0
    with pytest.raises(ric.RicError) as e:                   # the schedule is void
        ric.ric_compile(b.h, 8)
    assert e.value.code == ric.RIC_ESTATE
    b.close()


def test_move_of_shared_pages_without_caches(rt):
    ric, runner = rt
    b, *_ = make(rt, reqs=0, max_reqs=6)
    for i in range(5):
        ric.ric_add_request(b.h, i, [1] * 40, 40, 0, [50, 60, 70 + i])
    ric.ric_move_blocks(b.h, [60, 72, 50], [2, 3, 99], [], [], 0)
    tab = b.block_table().cpu().numpy()
    for i in range(5):
        assert list(tab[i, :3]) == [99, 2, 3 if i == 2 else 70 + i]
    refs = runner.block_refs(b).cpu().numpy()
    assert refs[99] == 5 and refs[2] == 5 and refs[50] == 0
    b.close()


@pytest.mark.parametrize("computed", [0, 1, 16, 33, 47, 48])
def test_fork_shares_full_pages_and_copies_the_partial_one(rt, computed):
    ric, runner = rt
    b, tables, _, toks, rng = make(rt, reqs=0, max_reqs=5)
    T = 50
    parent = np.arange(100, 100 + T).astype(np.int32)
    ric.ric_add_request(b.h, 7, parent, 20, 0, [11, 12, 13, 14], (0.7, 0.8, 1.3, 9))
    sampled = torch.tensor([777], dtype=torch.int32, device="cuda")
    ric.ric_append_sampled(b.h, [0], sampled.data_ptr(), 1)              # a token the host never saw
    kc, vc = caches(35, 100, 16, 64, 1)
    before = [c.clone() for c in kc + vc]
    shared, tail = computed // 16, computed % 16
    new = [40, 41] if tail else [40]
    row = runner.fork_request(b, 7, 8, T + 1, computed, new, kc, vc)
    assert row == 1 and ric.ric_row_of(b.h, 8) == 1
    cols = ric.ric_get_columns(b.h)
    got = read_rows_i32(b.workspace, cols.tokens, cols.token_stride, [row], T + 1)[0]
    assert list(got) == list(parent) + [777]
    got = read_rows_i32(b.workspace, cols.blocks, cols.block_stride, [row], shared + len(new))[0]
    assert list(got) == [11, 12, 13, 14][:shared] + new
    for c, old in zip(kc + vc, before):
        want = old.clone()
        if tail:
            want[40, :tail] = old[[11, 12, 13, 14][shared], :tail]
        assert torch.equal(c, want)
    one = lambda p, dt=torch.int32: runner._view_u8(b.workspace, p + 4 * row, 4).view(dt).item()
    assert (one(cols.num_tokens), one(cols.num_prompt), one(cols.num_computed), one(cols.num_blocks)) == \
        (T + 1, 20, computed, shared + len(new))
    assert one(cols.top_k) == 9 and one(cols.temperature, torch.float32) == np.float32(0.7)
    # the child is scheduled and compiled like any request
    cap = 16 * (shared + len(new))
    q = min(T + 1, cap) - computed
    ric.ric_schedule(b.h, [0, computed], [1, q])
    s = b.compile(1 + q)
    got = b.step_outputs(s)
    table = [11, 12, 13, 14][:shared] + new
    assert list(got["slot_mapping"][1:]) == [table[p // 16] * 16 + p % 16 for p in range(computed, computed + q)]
    assert list(got["input_ids"][1:]) == (list(parent) + [777])[computed:computed + q]
    b.close()


def test_forks_on_another_stream_then_attention(rt):
    """Two forks of one request, each writing its own next token: the shared
    prefix is read by both, the written rows by their owner alone."""
    ric, runner = rt
    from tests.ops_helpers import attention_reference, check_attention
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = runner.Batch(ric.make_config(max_num_reqs=4, max_model_len=128, block_size=16, max_blocks_per_req=8,
                                         max_num_batched_tokens=64, num_kv_blocks=40, null_block=0, staging_bytes=0))
        g = torch.Generator(device="cuda").manual_seed(4)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        kc, vc = [rnd(40, 16, 2, 64)], [rnd(40, 16, 2, 64)]
        ric.ric_add_request(b.h, 0, np.arange(41), 38, 40, [5, 6, 7])
        runner.fork_request(b, 0, 1, 41, 40, [20], kc, vc)
        runner.fork_request(b, 0, 2, 41, 40, [21], kc, vc, sampling=(0.1, 1.0, 1.0, 3))
        ric.ric_schedule(b.h, [40, 40, 40], [1, 1, 1])
        k, v, q = [rnd(3, 2, 64)], [rnd(3, 2, 64)], rnd(3, 8, 64)
        step = runner.compile_and_cache(b, 3, runner.KVSet(k, v, kc, vc, 256, 640))
        out = torch.zeros_like(q)
        runner.step_attention(b, step, q, kc[0], vc[0], out)
    side.synchronize()
    table = torch.tensor([[5, 6, 7], [5, 6, 20], [5, 6, 21]], dtype=torch.int32, device="cuda")
    for i, page in enumerate((7, 20, 21)):
        assert torch.equal(kc[0][page, 8], k[0][i]) and torch.equal(kc[0][page, :8], kc[0][7, :8])
    inp = dict(q=q, kc=kc[0], vc=vc[0], table=table, lens=[(1, 41)] * 3)
    want, tol = attention_reference(inp, scale=64 ** -0.5)
    check_attention(out, want, tol)
    b.close()
