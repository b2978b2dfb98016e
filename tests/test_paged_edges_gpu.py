"""Edges of the paged serving operators on the GPU."""
import ctypes

import pytest
import torch

import paged_attention_varlen_b200 as ala
import paged_ref
from test_paged_edges import carried_bound
from test_paged_gpu import BF, FP, _compare, _dev, _plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from paged_attention_varlen_b200 import build
    build.build()


def _graph(op):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op()
    return graph


# ---------------------------------------------------------------------------------------------- status

@pytest.mark.parametrize("lens", [[(1, 200), (1, 90)], [(60, 200), (40, 90)]])
def test_a_status_that_was_read_is_gone_from_what_is_captured_after_it(lens):
    c = paged_ref.make_case(lens, 4, 2, 64, BF, 16, 9, 10)
    op, out, lse = _plan(c)
    tables = op._keep[3]
    tables[0, 3] = -1
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0x10B
    tables.copy_(c["tables"])
    graph = _graph(op)
    for _ in range(2):
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert op.device_status() == 0
        _compare(c, out, lse)


@pytest.mark.parametrize("lens", [[(1, 200), (1, 90)], [(60, 200), (40, 90)]])
def test_binding_clears_the_status_of_a_loop_of_replays(lens):
    c = paged_ref.make_case(lens, 4, 2, 64, BF, 16, 9, 20)
    op, out, lse = _plan(c)
    op()
    graph = _graph(op)
    tables = op._keep[3]
    tables[0, 3] = -1
    graph.replay()
    torch.cuda.synchronize()
    assert op.device_status() == 0x10B
    tables.copy_(c["tables"])
    op.bind()
    out.fill_(7.0)
    lse.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    _compare(c, out, lse)


def test_binding_is_refused_on_a_stream_that_is_captured():
    c = paged_ref.make_case([(1, 40)], 4, 2, 64, BF, 16, 9, 25)
    op, out, lse = _plan(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError):
            op.bind()
        op()
    graph.replay()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    _compare(c, out, lse)


def test_an_execution_with_no_rows_clears_an_unbound_workspace():
    c = paged_ref.make_case([(0, 0), (0, 50)], 4, 2, 64, BF, 16, 9, 30)
    op, out, lse = _plan(c)
    ws = torch.full((op.workspace_size,), 0xA5, dtype=torch.uint8, device="cuda")
    stream, code = torch.cuda.current_stream().cuda_stream, ctypes.c_int32(-1)
    assert ala.lib().ala_paged_attention(ws.data_ptr(), op.workspace_size, op._handle, stream) == 0
    assert ala.lib().ala_workspace_status(op._handle, ws.data_ptr(), stream, ctypes.byref(code)) == 0
    assert code.value == 0


@pytest.mark.parametrize("lens,d", [([(1, 3000), (2, 900)], 128), ([(1, 40)] * 70, 64), ([(90, 2000), (1, 50)], 64), ([(70, 400)], 256),
                                    ([(150, 400)] + [(1, 70)] * 20, 128)])
def test_after_a_recorded_wait_nothing_is_written_until_the_workspace_is_bound_again(lens, d):
    # the code is put where a wait that ran out would leave it, and the counters as a cut item would
    c = paged_ref.make_case(lens, 8, 2, d, BF, 64, 9, 35 + d)
    op, out, lse = _plan(c)
    op.bind()
    header = op.workspace[:1024].view(torch.int32)
    header[0] = 0x105
    header[64:64 + 148] = 1
    op()
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (lse == 7.0).all()
    assert op.device_status() == 0x105
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    _compare(c, out, lse)
    assert (op.workspace[:1024] == 0).all()


# ---------------------------------------------------------------------------------------------- a norm without an epsilon

@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens", [[(2, 0), (5, 3), (1, 40)], [(60, 9), (1, 0)], [(200, 150), (3, 0)]])  # few rows, one block of rows, two
def test_rows_without_a_key_get_zero_under_a_norm_without_an_epsilon(lens, d):
    c = paged_ref.make_case(lens, 4, 2, d, BF, 16, 9, 60 + d, maps=2, norm=True)
    c["eps"] = 0.0
    op, out, _ = _plan(c)
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    keyless = torch.cat([torch.arange(n) + kv - n < 0 for n, kv in lens])
    assert keyless.any()
    got = out.cpu().double()
    assert (got[keyless] == 0).all()
    ref, _, tol, _ = paged_ref.attention(c)
    assert ((got - ref).abs() <= tol)[~keyless].all()


def test_values_of_zero_give_zero_under_a_norm_without_an_epsilon():
    # whole items and items that several CTAs share
    c = paged_ref.make_case([(1, 4000), (2, 70)], 4, 2, 64, BF, 16, 9, 70, maps=2, norm=True)
    c["eps"] = 0.0
    c["v"].zero_()
    op, out, _ = _plan(c)
    op()
    torch.cuda.synchronize()
    assert (out == 0).all()


# ---------------------------------------------------------------------------------------------- output over the query

@pytest.mark.parametrize("lens", [[(1, 40), (1, 5000), (2, 300)], [(140, 900), (3, 20)], [(200, 3000), (33, 50)]])
@pytest.mark.parametrize("maps,d", [(1, 64), (1, 128), (1, 256), (2, 32), (2, 64), (2, 128)])
def test_the_output_may_lie_on_a_dense_query(maps, d, lens):
    c = paged_ref.make_case(lens, 4, 2, d, BF, 16, 9, 100 + d, maps=maps)
    q = _dev(c["q"])
    common = [_dev(c[x]) for x in ("k", "v", "tables", "seq", "kv")]
    out = q.view(q.shape[0], 4, maps * d)
    if maps == 2:
        op, _ = ala.plan_paged_diff_attention(q, *common, _dev(c["lam"]), 9, 4, 2, c["scale"], out=out)
    else:
        op, _ = ala.plan_paged_attention(q, *common, 9, 4, 2, c["scale"], out=out)
    for _ in range(3):
        q.copy_(c["q"])
        op()
        torch.cuda.synchronize()
        assert op.device_status() == 0
        _compare(c, out, None)


# ---------------------------------------------------------------------------------------------- the remainder of P

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,heads,kv_heads,d,maps,mask", [
    ([(1, 60), (1, 33), (1, 128), (0, 0), (1, 7), (1, 300)], 8, 2, 64, 1, 9), ([(1, 60), (1, 33), (1, 130)], 16, 1, 128, 1, 0),
    ([(2, 60), (2, 33), (1, 64)], 8, 1, 256, 1, 9), ([(1, 60), (1, 33), (1, 128)], 4, 4, 80, 1, 4),
    ([(1, 60), (1, 33), (1, 128), (1, 7)], 4, 2, 64, 2, 9), ([(1, 60), (1, 40)], 16, 1, 32, 2, 0), ([(2, 60), (4, 40)], 4, 1, 128, 2, 9),
    ([(60, 70), (1, 33)], 4, 2, 64, 2, 9), ([(150, 160)], 4, 2, 32, 2, 9), ([(40, 90)], 2, 1, 128, 2, 0)])
def test_p_carries_what_its_rounding_drops(lens, heads, kv_heads, d, maps, mask, dtype, monkeypatch):
    # up to 16 rows of one map, and every difference of two: held to carried_bound
    c = paged_ref.make_case(lens, heads, kv_heads, d, dtype, 16, mask, 80 + d, maps=maps)
    c["scale"] /= 16  # small scores: their own errors are below those of P
    op, out, _ = _plan(c)
    op()
    torch.cuda.synchronize()
    ref, tol = carried_bound(c, monkeypatch)
    worst = ((out.cpu().double()[:len(ref)] - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"error {worst:.2f} times its bound"


# ---------------------------------------------------------------------------------------------- lengths that are cut

@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("shape,pad", [((1, 1, 2), 0), ((1, 1, 2), 90), ((70, 1, 90), 0), ((70, 1, 90), 14)])
# few rows, scanned in registers and by the CTA; many rows, alone and with a launch for few
def test_lengths_that_are_cut_spoil_their_own_rows_only(shape, pad, d):
    n0, n1, n2 = shape
    kv = (200, 90, 150)
    idle = [(0, 5)] * pad
    c = paged_ref.make_case([(n0, kv[0]), (n1, kv[1]), (n2, kv[2]), *idle], 8, 2, d, BF, 16, 9, 40 + d)
    c["tables"][c["tables"] < 0] = 0  # every entry may be read
    op, out, lse = _plan(c)
    total, big = sum(shape), 2 ** 31 - 1
    # (lengths as they lie in memory, as they count for packing, the sequences that are cut)
    for seq, keys, packed, cut in [
            ((n0, n1 + total, n2), kv, (n0, total - n0, 0), (1, 2)), ((-3, n1, n2), kv, (0, n1, n2), (0,)),
            ((n0, n1, n2), (-5, kv[1], kv[2]), (n0, n1, n2), (0,)), ((n0, n1, n2), (kv[0], big, kv[2]), (n0, n1, n2), (1,)),
            ((n0, n1, n2), (kv[0], -2 ** 31, kv[2]), (n0, n1, n2), (1,)), ((n0, n1, big), kv, (n0, n1, n2), (2,)),
            ((big, big, big), kv, (total, 0, 0), (0, 1, 2))]:
        op._keep[4].copy_(torch.tensor([*seq, *[0] * pad], dtype=torch.int32))
        op._keep[5].copy_(torch.tensor([*keys, *[5] * pad], dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        op()
        torch.cuda.synchronize()
        assert op.device_status() == 0x10C
        at, own = 0, torch.zeros(total, dtype=torch.bool)
        for b, n in enumerate(packed):
            own[at:at + n] = b not in cut
            at += n
        ref, lref, tol, ltol = paged_ref.attention({**c, "seq": torch.tensor([*packed, *[0] * pad])})
        own = own[:ref.shape[0]]
        assert ((out.cpu().double()[:len(own)] - ref).abs() <= tol)[own].all()
        assert ((lse.cpu().double()[:len(own)] - lref).abs() <= ltol)[own].all()
        assert (out[at:] == 7.0).all() and (lse[at:] == 7.0).all()
    op._keep[4].copy_(c["seq"])
    op._keep[5].copy_(c["kv"])
    op()
    torch.cuda.synchronize()
    assert op.device_status() == 0
    _compare(c, out, lse)
