"""Log probabilities, ranks, entropies and top alternatives against their
definition in 64 bits: types, vocabularies from one token to long odd ones,
alignments, ties, masked and broken rows, device counts, streams and graphs."""
import numpy as np
import pytest
import torch

from tests.ops_helpers import logprob_reference

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def runner():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ragged_input_compilation_amd import runner
    return runner


def compare(o, want, rows, vocab, label=""):
    """Ids and ranks are equal.  Float outputs: with d = x - m, the weight e^d is
    off by (|d| + 3) 2^-24 relative (the subtraction is off by 2^-24 |d|, its
    scaling and the exponential by 2^-22 together), a weight of relevance has
    |d| < 30, and the sums of up to vocab terms add (vocab / 256 + 16) 2^-24 (each
    lane adds its share, then the lanes are added): ln S is off by that much
    plus 2^-22 of its own size, the entropy by as much again per unit of |W / S|."""
    lp, rank, ent, ids, tlp = want
    assert torch.equal(o.rank[:rows].long(), rank.long()), label
    assert torch.equal(o.top_ids[:rows].long(), ids.long()), label
    rel = (40 + vocab / 256 + 16) * 2.0 ** -24 * 2
    for got, ref, name in ((o.logprob[:rows], lp, "logprob"), (o.entropy[:rows], ent, "entropy"),
                           (o.top_logprobs[:rows], tlp, "top")):
        got = got.double()
        # a difference past float32's range (two bfloat16 extremes are 6.8e38
        # apart, float32 ends at 3.4e38) is -inf in the float32 output
        ref = torch.where(ref < -torch.finfo(torch.float32).max, torch.full_like(ref, -INF), ref)
        same = (got == ref) | (got.isnan() & ref.isnan())
        ok = same | ((got - ref).abs() <= rel * (1 + ref.abs()) + 2.0 ** -21 * (ref.abs() + 12))
        assert ok.all(), f"{label} {name}: got {got[~ok][:4].tolist()} want {ref[~ok][:4].tolist()}"


def run(runner, x, t, k, label="", **kw):
    o = runner.token_logprobs(x, t, k, **kw)
    compare(o, logprob_reference(x, t, k), x.shape[0], x.shape[1], label)
    return o


def draw(rows, vocab, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((rows, vocab), generator=g, device="cuda") * spread).to(dtype)
    return x, torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,k", [
    (1, 1, 1), (3, 2, 2), (5, 7, 0), (4, 63, 5), (4, 64, 64), (2, 65, 64), (7, 1000, 20), (1, 32000, 5), (300, 4099, 3),
    (9, 50257, 20), (2, 152064, 64), (33, 128256, 1), (1, 1000003, 20), (2000, 513, 5)])
def test_shapes(runner, dtype, rows, vocab, k):
    x, t = draw(rows, vocab, dtype, seed=rows + vocab)
    run(runner, x, t, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_id(runner, dtype):
    x = torch.zeros((6, 5003), dtype=dtype, device="cuda")
    x[1] = -0.0
    x[1, ::3] = 0.0                               # -0 and +0 are one value
    x[2] = torch.arange(5003, device="cuda").remainder(4).to(dtype)
    x[3, 2500:] = 1.0
    x[4] = torch.arange(5003, device="cuda").div(64, rounding_mode="floor").to(dtype)     # ascending in steps
    x[5] = -x[4]
    t = torch.tensor([4000, 5002, 2, 2499, 1, 5002], dtype=torch.int32, device="cuda")
    run(runner, x, t, 64)
    run(runner, x[:, :1000], t.clamp(max=999), 10)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 70001])
def test_masked_and_broken_rows(runner, dtype, vocab):
    """-inf and the type's lowest value as masks, rows of nothing else, NaN and
    +inf, values whose differences overflow."""
    x, t = draw(12, vocab, dtype, seed=3)
    low = torch.finfo(dtype).min
    x[0, 1::2] = -INF
    x[1, 1::2] = low
    x[2] = -INF
    x[3] = low
    x[4] = -INF
    x[4, vocab - 1] = 3.0
    x[5, vocab // 2] = float("nan")
    x[6, 7] = INF
    x[7, 3] = float("nan")
    x[7, vocab - 2] = -float("nan")
    x[7, 9] = INF
    x[8] = torch.finfo(dtype).max
    x[9, ::2] = torch.finfo(dtype).max
    x[9, 1::2] = low
    x[10, :vocab - 1] = -INF
    t[0], t[4], t[5], t[6], t[7], t[10] = 1, 0, vocab // 2, 8, vocab - 2, vocab - 1
    run(runner, x, t, 20)


def test_descending_and_ascending_rows_keep_the_order(runner):
    """Orders that make every token a candidate when it is met."""
    for vocab in (4096, 100000):
        up = torch.linspace(-8, 8, vocab, device="cuda")
        x = torch.stack([up, up.flip(0), up.roll(17), up.abs()])
        t = torch.tensor([0, vocab - 1, 5, vocab // 2], dtype=torch.int32, device="cuda")
        run(runner, x, t, 64)
        run(runner, x.to(torch.bfloat16), t, 64)


def test_targets_outside_and_missing(runner):
    x, t = draw(5, 300, torch.bfloat16)
    t[0], t[2], t[4] = -1, 300, 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = run(runner, x, t, 4, dev_status=status.data_ptr())
    assert status.item() == 2
    assert o.rank.tolist()[0] == 0 and o.logprob.tolist()[0] == 0.0
    o = runner.token_logprobs(x, None, 4)
    want = logprob_reference(x, t, 4)
    assert torch.equal(o.top_ids.long(), want[3])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_strided_and_misaligned_rows(runner, dtype):
    base, t = draw(6, 9001, dtype, seed=8)
    for lo, hi in ((1, 8000), (3, 9001), (7, 7 + 515), (5, 6)):
        x = base[:, lo:hi]
        run(runner, x, t % (hi - lo), min(5, hi - lo), f"[{lo}:{hi}]")
    flat = base.reshape(-1)[1:]                       # one row that starts off any 4- or 16-byte boundary
    run(runner, flat[:9000].unsqueeze(0), t[:1] % 9000, 7)


@pytest.mark.parametrize("vocab", [700, 60000])
def test_device_count_leaves_the_rest(runner, vocab):
    x, t = draw(9, vocab, torch.bfloat16)
    want = logprob_reference(x, t, 3)
    for n, c in ((4, 4), (0, 0), (9, 50), (0, -3)):
        cnt = torch.tensor([c], dtype=torch.int32, device="cuda")
        o = runner.alloc_logprobs(9, vocab, 3)
        for z in (o.logprob, o.entropy, o.top_logprobs):
            z.fill_(-5.0)
        for z in (o.rank, o.top_ids):
            z.fill_(-5)
        runner.token_logprobs(x, t, 3, o, dev_count=cnt.data_ptr())
        compare(o, tuple(z[:n] for z in want), n, vocab)
        for z in (o.logprob, o.entropy, o.top_logprobs, o.rank, o.top_ids):
            assert (z[n:] == -5).all()


def test_outputs_of_many_rows_take_fewer(runner):
    """Few rows are cut into pieces that many rows are not."""
    x, t = draw(1024, 16500, torch.bfloat16, seed=3)
    o = runner.alloc_logprobs(1024, 16500, 5)
    want = logprob_reference(x, t, 5)
    for n in (1024, 1000, 600, 511, 2, 1):
        runner.token_logprobs(x[:n], t[:n], 5, o)
        compare(o, tuple(z[:n] for z in want), n, 16500, f"{n} rows")


@pytest.mark.parametrize("rows,vocab", [(3, 50257), (400, 2000)])
def test_stream_graph_and_equal_bits(runner, rows, vocab):
    sets = [draw(rows, vocab, torch.bfloat16, seed=s) for s in range(3)]
    x, t = sets[0][0].clone(), sets[0][1].clone()
    outs = [runner.alloc_logprobs(rows, vocab, 5) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        runner.token_logprobs(x, t, 5, outs[0])
    side.synchronize()
    compare(outs[0], logprob_reference(x, t, 5), rows, vocab)
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            runner.token_logprobs(x, t, 5, o)
        graphs.append(g)
    for a, b in sets * 2:
        x.copy_(a)
        t.copy_(b)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = runner.token_logprobs(x, t, 5)
        want = logprob_reference(x, t, 5)
        for o in outs:
            compare(o, want, rows, vocab)
            for name in ("logprob", "rank", "entropy", "top_ids", "top_logprobs"):
                assert torch.equal(getattr(o, name), getattr(eager, name)), name


def test_rows_past_4_gib(runner):
    """Row offsets that need more than 32 bits."""
    vocab, rows = 1 << 20, 2100
    x = torch.empty((rows, vocab), dtype=torch.bfloat16, device="cuda")
    x.fill_(-4.0)
    t = torch.zeros(rows, dtype=torch.int32, device="cuda")
    pick = [0, 1, 2047, 2048, 2099]
    y, ty = draw(len(pick), vocab, torch.bfloat16, seed=1)
    x[pick] = y
    t[pick] = ty
    o = runner.token_logprobs(x, t, 4)
    want = logprob_reference(y, ty, 4)
    part = type(o)(o.logprob[pick], o.rank[pick], o.entropy[pick], o.top_ids[pick], o.top_logprobs[pick], None)
    compare(part, want, len(pick), vocab)
