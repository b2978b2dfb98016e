"""The paged serving operators on the GPU against their plain 64-bit forms (paged_ref.py)."""
import random

import pytest
import torch

import paged_attention_varlen_b200 as ala
import paged_ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from paged_attention_varlen_b200 import build
    build.build()


def _dev(x):
    return None if x is None else x.cuda()


def _plan(c, lse=True, q=None):
    """(op, out, lse): outputs start out as a pattern that rows without a token must keep."""
    q = _dev(c["q"]) if q is None else q
    n, heads = q.shape[0], c["heads"]
    common = [_dev(c[x]) for x in ("k", "v", "tables", "seq", "kv")]
    if c["maps"] == 2:
        out = torch.full((n, heads, c["v"].shape[-1]), 7.0, dtype=q.dtype, device="cuda")
        op, out = ala.plan_paged_diff_attention(q, *common, _dev(c["lam"]), c["mask"], heads, c["kv_heads"], c["scale"],
                                                norm_weight=_dev(c["norm"]), norm_eps=c["eps"], out_scale=c["out_scale"],
                                                out=out)
        return op, out, None
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    l = torch.full((n, heads), 7.0, device="cuda") if lse else None
    op, out = ala.plan_paged_attention(q, *common, c["mask"], heads, c["kv_heads"], c["scale"], slopes=_dev(c["slopes"]),
                                       out=out, lse=l)
    return op, out, l


def _compare(c, out, lse):
    ref, lref, tol, ltol = paged_ref.attention(c)
    n = ref.shape[0]
    got = out.cpu().double()
    assert torch.isfinite(got[:n]).all()
    worst = ((got[:n] - ref).abs() / tol).max().item() if n else 0.0
    assert worst <= 1.0, f"error {worst:.2f} times its bound"
    assert (got[n:] == 7.0).all(), "rows behind the last sequence were written"
    if lse is not None:
        l = lse.cpu().double()
        empty = torch.isinf(lref)
        assert (l[:n][empty] == -float("inf")).all()
        worst = ((l[:n] - lref).abs() / ltol)[~empty].max().item() if (~empty).any() else 0.0
        assert worst <= 1.0, f"lse error {worst:.2f} times its bound"
        assert (l[n:] == 7.0).all()


def _check(c, **kw):
    op, out, lse = _plan(c, **kw)
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0, hex(op.device_status())
    _compare(c, out, lse)
    return op, out, lse


MIXED = [(1, 1), (1, 63), (1, 64), (1, 65), (0, 0), (3, 130), (1, 300), (0, 200), (70, 70), (33, 129), (200, 333)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("mask", [0, 3, 4, 5, 9])
def test_mixed_batch_of_every_mask(mask, dtype):
    _check(paged_ref.make_case(MIXED, 8, 2, 64, dtype, 32, mask, 10 + mask, tail=3))


@pytest.mark.parametrize("d", [8, 16, 40, 72, 80, 96, 112, 128, 136, 192, 256])
def test_head_sizes(d):
    _check(paged_ref.make_case(MIXED, 4, 2, d, FP if d % 16 else BF, 16, 9, 100 + d, tail=1))


@pytest.mark.parametrize("block", [16, 48, 64, 80, 128, 160, 256])
def test_page_sizes(block):
    _check(paged_ref.make_case(MIXED, 6, 2, 128, BF, block, 9, 200 + block))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (5, 5), (8, 1), (16, 1), (32, 2), (33, 1), (40, 8), (128, 1), (6, 3)])
def test_groups(heads, kv_heads):
    lens = [(1, 257), (2, 190), (0, 0), (1, 5), (9, 40), (130, 140)] if heads < 128 else [(1, 257), (5, 60), (1, 1)]
    _check(paged_ref.make_case(lens, heads, kv_heads, 64, BF, 16, 9, 300 + heads, tail=2))


@pytest.mark.parametrize("mask,d,dtype", [(9, 128, BF), (0, 64, FP), (5, 80, FP), (9, 256, BF), (4, 64, BF)])
def test_long_rows_are_split_over_the_grid_and_joined(mask, d, dtype):
    lens = [(1, 5000)] if d != 64 else [(1, 9001), (2, 17), (1, 3000)]
    _check(paged_ref.make_case(lens, 4, 1, d, dtype, 64, mask, 400 + d + mask))


@pytest.mark.parametrize("maps,d", [(1, 64), (1, 128), (2, 64)])
def test_many_tiles_for_every_cta(maps, d):
    # more tiles than CTAs, several items each: whole items, cut ones, and a running max that keeps growing
    g = torch.Generator().manual_seed(1)
    lens = [(1, int(torch.randint(1500, 4000, (1,), generator=g))) for _ in range(12)] + [(3, 2500), (40, 2000)]
    c = paged_ref.make_case(lens, 8, 4, d, BF, 64, 9, 450 + d, maps=maps)
    op, out, lse = _check(c)
    first = out.clone()
    for _ in range(20):
        op()
        assert torch.equal(out, first)
    # keys that grow along the sequence, so that the output is rescaled again and again
    for b, (_, kv) in enumerate(lens):
        blocks = c["tables"][b, :-(-kv // 64)].long()
        grow = (torch.arange(len(blocks) * 64, dtype=torch.float32).view(-1, 64, 1, 1) / kv * 30).to(BF)
        c["k"][blocks] = c["k"][blocks] * grow
    _check(c)


def _grow(c, lens, backwards, block):
    """Keys that grow along (or against) the sequence, so that the running maximum moves again and again."""
    for b, (_, kv) in enumerate(lens):
        blocks = c["tables"][b, :-(-kv // block)].long()
        at = torch.arange(len(blocks) * block, dtype=torch.float32).view(-1, block, 1, 1) / max(kv, 1)
        c["k"][blocks] = c["k"][blocks] * ((1 - at).clamp(min=0) if backwards else at).mul(30).to(c["k"].dtype)


@pytest.mark.parametrize("backwards", [False, True])
@pytest.mark.parametrize("lens,heads,kv_heads,d,maps", [
    ([(1, 1300), (1, 700)], 4, 1, 128, 1), ([(2, 1300), (1, 64)], 12, 2, 64, 1), ([(5, 900)], 5, 1, 80, 1), ([(1, 900)], 32, 1, 256, 1),
    ([(40, 700), (1, 300)], 4, 2, 128, 1), ([(40, 700), (33, 500)], 4, 2, 64, 1), ([(50, 600)], 2, 1, 256, 1),
    ([(300, 900), (1, 200)], 4, 2, 128, 1), ([(1, 700), (2, 300)], 4, 1, 64, 2), ([(150, 600)], 4, 2, 32, 2), ([(60, 400)], 2, 1, 128, 2)])
def test_a_running_maximum_that_keeps_moving(lens, heads, kv_heads, d, maps, backwards):
    c = paged_ref.make_case(lens, heads, kv_heads, d, BF, 64, 9, 470 + d, maps=maps)
    _grow(c, lens, backwards, 64)
    _check(c)


@pytest.mark.parametrize("d,maps", [(64, 1), (128, 1), (256, 1), (32, 2), (64, 2), (128, 2)])
def test_decoding_rows_beside_chunks(d, maps):
    # sequences of few rows and of many in one batch: two launches share the work
    rng = random.Random(d)
    lens = [(1, rng.randint(1, 900)) for _ in range(9)] + [(150, 400), (0, 70), (3, 333), (200, 200), (40, 1000), (1, 2)]
    _check(paged_ref.make_case(lens, 8, 2, d, BF, 32, 9, 480 + d, maps=maps, tail=3, norm=True))


@pytest.mark.parametrize("n,kv", [(1, 1), (1, 2), (2, 2), (127, 127), (128, 128), (129, 640), (1, 128), (1, 129)])
def test_single_sequences(n, kv):
    for d in (64, 128, 256):
        _check(paged_ref.make_case([(n, kv)], 2, 1, d, BF, 16, 9, 500 + n + kv))


def test_rows_without_a_key():
    # kvSeqLen 0, and fewer keys than new tokens: the first tokens see nothing and get 0 and -inf
    for mask in (0, 3, 4, 5, 9):
        c = paged_ref.make_case([(2, 0), (5, 3), (1, 40), (140, 9), (1, 0)], 4, 2, 64, BF, 16, mask, 600 + mask)
        _, out, lse = _check(c)
        assert (out[:2] == 0).all() and (mask == 0 or (out[2:4] == 0).all())
    c = paged_ref.make_case([(2, 0), (5, 3), (1, 40)], 4, 2, 32, BF, 16, 9, 650, maps=2, norm=True)
    _, out, _ = _check(c)
    assert (out[:4] == 0).all()


@pytest.mark.parametrize("lens", [[(1, 40), (1, 5000), (2, 300)], [(140, 900), (3, 20)], [(200, 30000)]])
@pytest.mark.parametrize("maps,d", [(1, 64), (1, 128), (1, 256), (2, 32), (2, 64), (2, 128)])
def test_a_query_with_a_nan_spoils_its_own_row_only(maps, d, lens):
    c = paged_ref.make_case(lens, 4, 2, d, BF, 16, 9, 655 + d, maps=maps)
    q, n = c["q"].cuda(), c["q"].shape[0]
    bad = [(0, 1), (n - 1, 2), (n // 2, 3)]  # (token, head), of one map
    for t, h in bad:
        q[t, maps * h, 5] = float("nan")
    op, out, lse = _plan(c, q=q)
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    ref, lref, tol, ltol = paged_ref.attention(c)
    good = torch.ones(n, 4, dtype=torch.bool)
    for t, h in bad:
        good[t, h] = False
    got = out.cpu().double()
    assert got[~good].isnan().all()
    assert ((got[good] - ref[good]).abs() <= tol[good]).all()
    if lse is not None:
        l = lse.cpu().double()
        assert l[~good].isnan().all()
        assert ((l[good] - lref[good]).abs() <= ltol[good]).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    c = paged_ref.make_case([(1, 200), (40, 90)], 4, 2, 64, FP, 16, 9, 660)
    c["scale"] = scale
    _check(c)


def test_more_sequences_than_threads():
    rng = random.Random(5)
    lens = [(rng.choice([0, 1, 1, 2]), rng.randint(2, 40)) for _ in range(1100)] + [(3, 700)] + [(0, 0)] * 30
    _check(paged_ref.make_case(lens, 2, 1, 64, BF, 16, 9, 670, tail=5))


def test_nothing_to_do():
    for lens, tail in (([], 0), ([(0, 0), (0, 50)], 0), ([(0, 0), (0, 50)], 4)):
        c = paged_ref.make_case(lens, 4, 2, 64, BF, 16, 9, 680, tail=tail)
        op, out, lse = _plan(c)
        op()
        torch.cuda.synchronize()
        assert (out == 7.0).all() and (lse == 7.0).all() and op.device_status() == 0


def test_queries_sliced_from_a_fused_projection():
    c = paged_ref.make_case(MIXED, 4, 2, 64, BF, 32, 9, 690)
    fused = torch.full((c["q"].shape[0], 512), float("nan"), dtype=BF, device="cuda")
    fused[:, 128:384] = c["q"].flatten(1).cuda()
    op, out, lse = _plan(c, q=fused[:, 128:384].view(-1, 4, 64))
    op()
    _compare(c, out, lse)


@pytest.mark.parametrize("d", [8, 16, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_differential_head_sizes(d, norm):
    _check(paged_ref.make_case(MIXED, 4, 2, d, BF if d % 32 else FP, 16, 9, 700 + d, maps=2, tail=3, norm=norm))


@pytest.mark.parametrize("heads,kv_heads,mask", [(1, 1, 9), (3, 1, 0), (16, 4, 9), (64, 1, 9), (20, 1, 0), (5, 5, 9)])
def test_differential_groups(heads, kv_heads, mask):
    lens = [(1, 257), (2, 190), (0, 0), (1, 5), (9, 40), (1, 4000), (70, 140)] if heads < 64 else [(1, 257), (5, 60)]
    _check(paged_ref.make_case(lens, heads, kv_heads, 64, BF, 16, mask, 800 + heads, maps=2, norm=heads % 2 == 0))


@pytest.mark.parametrize("d", [16, 24, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads,new", [(2, 1, 1), (8, 1, 1), (12, 1, 1), (16, 1, 1), (6, 3, 2), (8, 2, 4), (4, 4, 9)])
def test_differential_few_rows(heads, kv_heads, new, d):
    # 4 to 32 rows of a kv head, whole items and cut ones, the norm and none
    lens = [(new, 2000), (1, 150), (new, 333), (0, 9), (new, max(new, 5))]
    _check(paged_ref.make_case(lens, heads, kv_heads, d, FP if d == 32 else BF, 32, 9, 850 + d + heads, maps=2, norm=d != 64, tail=2))


@pytest.mark.parametrize("mask", [0, 3, 4, 5, 9])
@pytest.mark.parametrize("heads,kv_heads,new,d", [(2, 2, 1, 64), (16, 1, 1, 128), (32, 1, 1, 64), (10, 2, 5, 80), (4, 1, 8, 128), (6, 2, 3, 40)])
def test_few_rows(heads, kv_heads, new, d, mask):
    lens = [(new, 2000), (1, 150), (new, 333), (0, 9), (new, max(new, 5))]
    _check(paged_ref.make_case(lens, heads, kv_heads, d, FP if d == 80 else BF, 32, mask, 870 + d + heads, tail=2))


@pytest.mark.parametrize("d", [136, 192, 256])
def test_few_rows_of_large_heads(d):
    for heads, kv_heads, new in ((4, 2, 1), (16, 1, 1), (8, 1, 4)):
        _check(paged_ref.make_case([(new, 1500), (new, 70), (1, 300)], heads, kv_heads, d, BF, 64, 9, 890 + d, tail=1))


def test_few_rows_in_a_batch_too_large_for_one_scan():
    # more than 64 sequences, more than the threads of a CTA, single tokens: every CTA scans the batch in steps
    rng = random.Random(9)
    lens = [(1, rng.choice([1, 2, 40, 129, 300])) for _ in range(700)] + [(0, 5)] * 3
    _check(paged_ref.make_case(lens, 4, 2, 64, BF, 16, 9, 895))


def test_one_plan_serves_changing_lengths_and_a_captured_graph():
    c = paged_ref.make_case([(1, 900), (2, 500), (1, 40), (60, 300)], 8, 2, 64, BF, 16, 9, 900, tail=10)
    op, out, lse = _plan(c)
    seq, kv = op._keep[4], op._keep[5]
    first_seq, first_kv = c["seq"].clone(), c["kv"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # captured before any execution: no binding
        op()
    for lens in ([(1, 900), (2, 500), (1, 40), (60, 300)], [(0, 900), (1, 3), (40, 40), (1, 1)], [(30, 900), (2, 2), (0, 0), (3, 300)]):
        c["seq"], c["kv"] = (torch.tensor(x, dtype=torch.int32) for x in zip(*lens))
        for run in (op, graph.replay):
            seq.copy_(c["seq"])
            kv.copy_(c["kv"])
            out.fill_(7.0)
            lse.fill_(7.0)
            run()
            torch.cuda.synchronize()
            _compare(c, out, lse)
    assert op.device_status() == 0
    seq.copy_(first_seq)
    kv.copy_(first_kv)
    op()
    again = out.clone()
    op()
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_two_ops_on_two_streams_and_another_stream_than_the_current():
    cases = [paged_ref.make_case([(1, 3000), (1, 700), (90, 400)], 8, 2, 128, BF, 64, 9, 910 + i) for i in range(2)]
    plans = [_plan(c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        plans[0][0](streams[0])
        with torch.cuda.stream(streams[1]):
            plans[1][0]()
    torch.cuda.synchronize()
    for c, (op, out, lse) in zip(cases, plans):
        assert op.device_status() == 0
        _compare(c, out, lse)


def test_bad_blocks_and_lengths_are_reported_and_read_nothing():
    c = paged_ref.make_case([(1, 200), (1, 90)], 4, 2, 64, BF, 16, 9, 920)
    op, out, lse = _plan(c)
    tables, seq, kv = op._keep[3], op._keep[4], op._keep[5]
    for bad in (-1, c["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        tables[0, 3] = bad
        op()
        torch.cuda.synchronize()
        assert op.device_status() == 0x10B
        assert torch.isfinite(out).all()
        ref = paged_ref.attention(c)
        assert ((out[1].cpu().double() - ref[0][1]).abs() <= ref[2][1]).all()  # the other sequence is untouched
    tables.copy_(c["tables"])
    for s, k in (([1, 5], [200, 90]), ([-3, 1], [200, 90]), ([1, 1], [-5, 90]), ([1, 1], [2 ** 31 - 1, 90]), ([2 ** 31 - 1, 2 ** 31 - 1], [200, 90])):
        seq.copy_(torch.tensor(s))
        kv.copy_(torch.tensor(k))
        op()
        torch.cuda.synchronize()
        assert op.device_status() in (0x10C, 0x10B)  # keys past the cache's table also meet its -1 entries
    seq.copy_(c["seq"])
    kv.copy_(c["kv"])
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    _compare(c, out, lse)


@pytest.mark.parametrize("lens,d", [([(1, 3000), (2, 900)], 128), ([(90, 400), (1, 50)], 64)])
def test_an_unbound_workspace_may_hold_anything(lens, d):
    c = paged_ref.make_case(lens, 8, 2, d, BF, 64, 9, 930 + d)
    op, out, lse = _plan(c)
    ws = torch.full((op.workspace_size,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out.fill_(7.0)
        assert ala.lib().ala_paged_attention(ws.data_ptr(), op.workspace_size, op._handle, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        _compare(c, out, lse)
    # bound by hand, and unbound again
    assert ala.lib().ala_op_bind_workspace(op._handle, ws.data_ptr(), op.workspace_size, None) == 0
    assert ala.lib().ala_paged_attention(ws.data_ptr(), op.workspace_size, op._handle, torch.cuda.current_stream().cuda_stream) == 0
    assert ala.lib().ala_op_bind_workspace(op._handle, None, 0, None) == 0
    torch.cuda.synchronize()
    _compare(c, out, lse)


@pytest.mark.parametrize("n", [1, 150])
def test_rows_past_four_gigabytes_of_cache(n):
    # a cache of 5 GiB whose last pages hold the sequence; what lies before them is never touched
    block, heads, d = 64, 8, 128
    blocks = (5 << 30) // (block * heads * d * 2)
    small = paged_ref.make_case([(n, 300)], 16, heads, d, BF, block, 9, 940)
    k = torch.empty(blocks, block, heads, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    # the rows go in through the write, slot by slot
    used = small["tables"][0, :5].long()
    far = torch.arange(blocks - 5, blocks)
    slots = torch.cat([b * block + torch.arange(block) for b in far])[:300].to(torch.int32).cuda()
    rows = lambda x: x[used].flatten(0, 1)[:300].contiguous().cuda()  # noqa: E731
    ala.paged_write(rows(small["k"]), rows(small["v"]), slots, k, v)
    tables = far.to(torch.int32).view(1, -1).cuda()
    out = torch.full((n, 16, d), 7.0, dtype=BF, device="cuda")
    op, _ = ala.plan_paged_attention(small["q"].cuda(), k, v, tables, small["seq"].cuda(), small["kv"].cuda(), 9, 16, heads,
                                     small["scale"], out=out)
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    _compare(small, out, None)


# ---------------------------------------------------------------------------------------------- step and write

def _step_case(rng, batch, width, block, ended=True):
    room = width * block  # keys that a request's table row holds
    ctx = [rng.randint(0, room // 2) for _ in range(batch)]
    seq = [min(room - c, rng.choice([0, 1, 1, 2, rng.randint(0, 3 * block)])) for c in ctx]
    done = [int(ended and rng.random() < 0.2) for _ in range(batch)]
    held = [-(-c // block) for c in ctx]
    want = sum(-(-((0 if e else c) + n) // block) for c, n, e in zip(ctx, seq, done))
    blocks = sum(held) + want + 5
    perm = list(range(blocks))
    rng.shuffle(perm)
    tables = [[perm.pop() for _ in range(h)] + [-1] * (width - h) for h in held]
    count = len(perm)
    return seq, ctx, done, tables, perm + [-7] * (blocks - count), count, block, sum(seq) + rng.randint(0, 40)


def _run_step(seq, ctx, done, tables, free, count, block, n_tokens, in_place=False):
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dseq, dctx, ddone, dtab, dfree, dcount = t(seq), t(ctx), t(done), t(tables).view(len(seq), -1), t(free), t([count])
    kw = dict(kv_seq_len=dctx, free_count_out=dcount) if in_place else {}
    out = ala.paged_step(dseq, dctx, dtab, dfree, dcount, block, n_tokens, finished=ddone if any(done) else None, **kw)
    torch.cuda.synchronize()
    return out, dtab.tolist(), dfree.tolist()


@pytest.mark.parametrize("batch,width,block", [(1, 1, 16), (1, 40, 1), (2, 9, 3), (33, 20, 16), (257, 12, 64), (1025, 9, 16),
                                               (3000, 7, 5), (8192, 2, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(batch, width, block, in_place):
    rng = random.Random(batch)
    for _ in range(3):
        args = _step_case(rng, batch, width, block)
        want = paged_ref.step(*args)
        assert not isinstance(want, int)
        out, tables, free = _run_step(*args, in_place=in_place)
        assert out.status.item() == 0
        kv, count, cu, slots, positions, wtables, wfree = want
        assert out.kv_seq_len.tolist() == kv and out.free_count.item() == count and out.cu_seq_len.tolist() == cu
        assert out.slot_mapping.tolist() == slots and out.positions.tolist() == positions
        assert tables == wtables and free == wfree


@pytest.mark.parametrize("batch", [63, 64, 65])
@pytest.mark.parametrize("tokens", [1000, 1024, 1025, 1500])
def test_step_with_one_block_of_threads_and_with_many(batch, tokens):
    rng = random.Random(batch * tokens)
    seq, *rest, n_tokens = _step_case(rng, batch, 40, 16)
    assert sum(seq) <= n_tokens
    n_tokens = max(tokens, sum(seq))
    want = paged_ref.step(seq, *rest, n_tokens)
    out, tables, free = _run_step(seq, *rest, n_tokens)
    assert out.status.item() == 0
    got = [out.kv_seq_len.tolist(), out.free_count.item(), out.cu_seq_len.tolist(), out.slot_mapping.tolist(),
           out.positions.tolist(), tables, free]
    assert got == list(want)


def test_step_that_cannot_be_served_changes_nothing():
    rng = random.Random(1)
    for batch in (5, 1500):
        seq, ctx, done, tables, free, count, block, n = _step_case(rng, batch, 10, 16)
        seq[0], seq[1], ctx[1] = 3, 40, 0  # request 1 needs blocks
        n = sum(seq) + 3
        bad = [(dict(seq=[-1] + seq[1:]), 1), (dict(seq=[161] + seq[1:]), 1), (dict(ctx=[161] + ctx[1:]), 1),
               (dict(seq=[2 ** 31 - 1] * batch), 1), (dict(ctx=[-2 ** 31] + ctx[1:]), 1), (dict(n=sum(seq) - 1), 2),
               (dict(count=-1), 3), (dict(count=len(free) + 1), 3), (dict(count=0, done=[0] * batch), 4)]
        for change, code in bad:
            a = dict(seq=seq, ctx=ctx, done=done, tables=tables, free=free, count=count, block=block, n=n)
            a.update(change)
            assert paged_ref.step(*a.values()) == code
            for in_place in (False, True):
                out, t, f = _run_step(*a.values(), in_place=in_place)
                assert out.status.item() == code
                assert t == tables and f == free and out.kv_seq_len.tolist() == a["ctx"]
                assert out.free_count.item() == a["count"] and out.cu_seq_len.tolist() == [0] * (batch + 1)
                assert out.slot_mapping.tolist() == [-1] * a["n"] and out.positions.tolist() == [0] * a["n"]


def test_step_reports_a_block_outside_the_cache():
    out, _, _ = _run_step([1, 1], [20, 3], [0, 0], [[5, 99], [2, -1]], list(range(8)), 4, 16, 2)
    assert out.status.item() == ala.STEP_BAD_BLOCK and out.slot_mapping.tolist() == [-1, 2 * 16 + 3]
    out, _, _ = _run_step([1], [16], [0], [[5, -1]], [0, 1, 2, -9], 4, 16, 1)
    assert out.status.item() == ala.STEP_BAD_BLOCK and out.slot_mapping.tolist() == [-1]


@pytest.mark.parametrize("tokens,row,vrow,dtype,pad", [
    (1, (8, 128), (8, 128), BF, 0), (37, (2, 64), (2, 64), FP, 256), (300, (1, 512), (1, 64), BF, 0), (50, (1, 5), (1, 3), BF, 1),
    (9, (3, 7), None, torch.float32, 2), (64, (1, 512), (1, 64), torch.int8, 0), (4097, (1, 16), (1, 16), torch.float32, 16),
    (20, (16, 256), (16, 256), torch.float32, 0), (3, (40, 250), (1, 1), FP, 3)])
def test_write(tokens, row, vrow, dtype, pad):
    g = torch.Generator().manual_seed(tokens)
    block, blocks = 16, tokens // 16 + 4

    def rows(shape, scale=100):
        return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()

    slots = torch.randperm(blocks * block, generator=g)[:tokens].to(torch.int32)
    if tokens > 5:
        slots[1], slots[4] = -1, blocks * block  # skipped
        slots[2] = -2 ** 31
    kc = rows((blocks, block, *row))
    vc = None if vrow is None else rows((blocks, block, *vrow))
    nk, nv = row[0] * row[1], 0 if vrow is None else vrow[0] * vrow[1]
    fused = rows((tokens, nk + nv + pad))
    key = fused[:, pad:pad + nk].view(tokens, *row)
    value = None if vrow is None else fused[:, pad + nk:].view(tokens, *vrow)
    want = [kc.clone(), None if vc is None else vc.clone()]
    for w, x in zip(want, (key, value)):
        if w is not None:
            for t, s in enumerate(slots.tolist()):
                if 0 <= s < blocks * block and (t < 50 or t > tokens - 50):
                    w.flatten(0, 1)[s] = x[t]
            live = (slots >= 0) & (slots < blocks * block)
            w.flatten(0, 1)[slots[live].long().cuda()] = x[live.cuda()]
    ala.paged_write(key, value, slots.cuda(), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, want[0]) and (vc is None or torch.equal(vc, want[1]))


def test_write_of_nothing():
    kc = torch.ones(2, 16, 8, device="cuda")
    ala.paged_write(torch.zeros(0, 8, device="cuda"), None, torch.zeros(0, dtype=torch.int32, device="cuda"), kc, None)
    torch.cuda.synchronize()
    assert (kc == 1).all()


# ---------------------------------------------------------------------------------------------- together

@pytest.mark.parametrize("maps", [1, 2])
def test_a_serving_loop_in_one_captured_graph(maps):
    """Requests join, decode, end and are replaced: one graph of step, write and attention serves every step, its
    state on the device.  Each step is compared with attention over the keys that the host kept."""
    heads, kv_heads, d, block, batch, width, n_tokens, dtype = 4, 2, 32, 16, 6, 8, 80, BF
    rng, g = random.Random(3), torch.Generator().manual_seed(3)
    cap = batch * width
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    seq, ctx, done, count = z(batch), z(batch), z(batch), torch.tensor([cap], dtype=torch.int32, device="cuda")
    tables, free = torch.full((batch, width), -1, dtype=torch.int32, device="cuda"), torch.randperm(cap, generator=g).int().cuda()
    qw, kw, vw = maps * heads * d, maps * kv_heads * d, kv_heads * maps * d
    fused = torch.zeros(n_tokens, qw + kw + vw, dtype=dtype, device="cuda")
    q = fused[:, :qw].view(n_tokens, maps * heads, d)
    key, value = fused[:, qw:qw + kw].view(n_tokens, maps * kv_heads, d), fused[:, qw + kw:].view(n_tokens, kv_heads, maps * d)
    kc = torch.full((cap, block, maps * kv_heads, d), float("nan"), dtype=dtype, device="cuda")
    vc = torch.full((cap, block, kv_heads, maps * d), float("nan"), dtype=dtype, device="cuda")
    step, out = ala.plan_paged_step(seq, ctx, tables, free, count, block, n_tokens, finished=done, kv_seq_len=ctx, free_count_out=count)
    write = ala.plan_paged_write(key, value, out.slot_mapping, kc, vc)
    lam = torch.tensor([0.1, 0.5, 0.8, 0.3])
    result = torch.full((n_tokens, heads, maps * d), 7.0, dtype=dtype, device="cuda")
    if maps == 1:
        attend, _ = ala.plan_paged_attention(q, kc, vc, tables, seq, ctx, 9, heads, kv_heads, 0.2, out=result)
    else:
        attend, _ = ala.plan_paged_diff_attention(q, kc, vc, tables, seq, ctx, lam.cuda(), 9, heads, kv_heads, 0.2, out=result)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        write()
        attend()
    held = [[] for _ in range(batch)]  # (k, v) rows of each request, on the host
    for it in range(12):
        ended = [int(bool(h) and (len(h) > 90 or rng.random() < 0.2)) for h in held]
        new = []
        for b in range(batch):
            if ended[b]:
                held[b] = []
            new.append(rng.choice([0, rng.randint(1, 30)]) if not held[b] else 1 if rng.random() < 0.8 else 3)
        while sum(new) > n_tokens:
            new[new.index(max(new))] = 0
        data = torch.randn(fused.shape, generator=g).to(dtype)
        fused.copy_(data)
        seq.copy_(torch.tensor(new))
        done.copy_(torch.tensor(ended))
        result.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert out.status.item() == 0 and attend.device_status() == 0
        at = 0
        for b in range(batch):
            for t in range(at, at + new[b]):
                held[b].append((data[t, qw:qw + kw].view(-1, d), data[t, qw + kw:].view(kv_heads, -1)))
            at += new[b]
        assert ctx.tolist() == [len(h) for h in held]
        # the same batch laid out by the host, one page a request
        c = dict(q=data[:, :qw].view(n_tokens, -1, d), seq=torch.tensor(new), kv=torch.tensor([len(h) for h in held]), heads=heads,
                 kv_heads=kv_heads, mask=9, scale=0.2, maps=maps, slopes=None, lam=lam, norm=None, eps=0.0, out_scale=1.0,
                 tables=torch.arange(batch).view(-1, 1))
        c["k"], c["v"] = torch.zeros(batch, 256, maps * kv_heads, d, dtype=dtype), torch.zeros(batch, 256, kv_heads, maps * d, dtype=dtype)
        for b, h in enumerate(held):
            for i, (k, v) in enumerate(h):
                c["k"][b, i], c["v"][b, i] = k, v
        _compare(c, result, None)
    used = sum(-(-len(h) // block) for h in held)
    assert count.item() == cap - used
