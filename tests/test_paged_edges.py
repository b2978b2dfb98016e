"""Calls of the paged serving operators that are refused on the host, or decided there, without a GPU."""
import ctypes

import pytest
import torch

import paged_attention_varlen_b200 as ala
import paged_ref


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_attention_varlen_b200 import build
    build.build()


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _aligned(*shape, dtype=torch.bfloat16):
    n = 1
    for s in shape:
        n *= s
    buf = torch.zeros(n + 64, dtype=dtype)
    at = -(buf.data_ptr() % 64) % 64 // buf.element_size()
    return buf[at:at + n].view(shape)


# ---------------------------------------------------------------------------------------------- host tensors

class _Stream:
    cuda_stream = 0


def _cpu_calls():
    """The four planned calls over tensors in host memory (planning them is allowed)."""
    q, kc = _aligned(3, 4, 64), _aligned(6, 16, 2, 64)
    yield ala.plan_paged_step(_i32(3), _i32(3), _i32(3, 4), _i32(6), _i32(1), 16, 5)[0]
    yield ala.plan_paged_write(q[:, :2], None, _i32(3), kc, None)
    yield ala.plan_paged_attention(q, kc, kc, _i32(3, 4), _i32(3), _i32(3), 9, 4, 2, 0.125)[0]
    yield ala.plan_paged_diff_attention(_aligned(3, 4, 32), _aligned(6, 16, 2, 32), _aligned(6, 16, 1, 64), _i32(3, 4), _i32(3), _i32(3),
                                        torch.zeros(2), 9, 2, 1, 0.125)[0]


@pytest.mark.parametrize("stream", [None, _Stream()])
@pytest.mark.parametrize("which", range(4))
def test_calls_over_host_tensors_launch_nothing(which, stream, monkeypatch):
    launched = []

    def stub(*args):
        launched.append(args)
        return 0

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    call = list(_cpu_calls())[which]
    setattr(call, "_function" if isinstance(call, ala.PagedCall) else "_execute", stub)
    with pytest.raises(ValueError):
        call(stream)
    assert not launched


# ---------------------------------------------------------------------------------------------- sizes

def _described(x, *shape):
    """x's memory under another shape."""
    t = ala.tensor(x)
    t.ndim = len(shape)
    for i, n in enumerate(shape):
        t.dims[i] = n
    return t


@pytest.mark.parametrize("heads,d", [(1 << 32, 1 << 32), (1 << 39, 1 << 39), (1 << 31, 1 << 33), (1 << 20, 1 << 20)])
def test_rows_whose_elements_cannot_be_counted_are_refused(heads, d):
    # products of two dims of up to 2^40 pass 64 bits, some of them to a row of 0 elements
    x, L, b = torch.zeros(64), ala.lib(), ctypes.byref
    rows, cache, slots = _described(x, 4, heads, d), _described(x, 3, 16, heads, d), ala.tensor(_i32(4))
    assert L.ala_paged_write(b(rows), 0, None, 0, b(slots), b(cache), None, None) == 2
    q, half, out = _aligned(4, 8, 64), _aligned(64), _aligned(4, 8, 64)
    ws, h = ctypes.c_uint64(0), ctypes.c_void_p(0)
    wide = _described(half, 3, 16, heads, d)
    st = L.ala_paged_attention_get_workspace_size(b(ala.tensor(q)), 0, b(wide), b(wide), b(ala.tensor(_i32(2, 4))), b(ala.tensor(_i32(2))),
                                                  b(ala.tensor(_i32(2))), None, 9, 8, 2, 0.1, b(ala.tensor(out)), None, b(ws), b(h))
    assert st == 2 and not h.value


# ---------------------------------------------------------------------------------------------- shared memory

@pytest.mark.parametrize("which", ["caches", "caches overlap", "key and its cache", "value and the key's cache", "slots"])
def test_a_write_whose_tensors_share_memory_is_refused(which):
    cache = torch.zeros(7, 16, 8)
    rows = torch.zeros(4, 8)
    a = dict(key=rows, value=torch.zeros(4, 8), key_cache=cache[:3], value_cache=cache[3:6], slots=_i32(4))
    a.update({"caches": dict(value_cache=cache[:3]), "caches overlap": dict(value_cache=cache[2:5]),
              "key and its cache": dict(key=cache[2, 12:]), "value and the key's cache": dict(value=cache[0, :4]),
              "slots": dict(slots=cache[1, 3, 4:].view(torch.int32))}[which])
    ts = [ala.tensor(a[x]) for x in ("key", "value", "slots", "key_cache", "value_cache")]
    r = [ctypes.byref(t) for t in ts]
    assert ala.lib().ala_paged_write(r[0], 0, r[1], 0, r[2], r[3], r[4], None) == 4, ala.lib().ala_last_error().decode()


def test_a_write_may_take_rows_that_lie_between_others():
    # key and value slices of one fused buffer, and the other half of the caches' storage, share no element
    fused, cache = torch.zeros(4, 32), torch.zeros(6, 16, 8)
    ts = [ala.tensor(x) for x in (fused[:0, :8], fused[:0, :8], _i32(0), cache[:3], cache[3:])]
    for t, at in zip(ts, (0, 32)):
        t.data, t.dims[0] = fused.data_ptr() + at, 0
    r = [ctypes.byref(t) for t in ts]
    assert ala.lib().ala_paged_write(r[0], 32, r[1], 32, r[2], r[3], r[4], None) == 0


def _flat(n, dtype=torch.bfloat16):
    return _aligned(n, dtype=dtype)


@pytest.mark.parametrize("which", ["query, shifted", "query, strided", "key", "value", "tables", "lengths", "lse", "lse on lengths", "slopes"])
def test_attention_whose_outputs_share_memory_is_refused(which):
    n, heads, d = 10, 8, 64
    size, buf = n * heads * d, _flat(2 * 6 * 16 * 2 * 64 + 64)
    q, out, kc, vc = _flat(size).view(n, heads, d), _flat(size).view(n, heads, d), _aligned(6, 16, 2, d), _aligned(6, 16, 2, d)
    a = dict(q=q, k_cache=kc, v_cache=vc, block_tables=_i32(3, 4), seq_len=_i32(3), kv_seq_len=_i32(3), mask_type=9, heads=heads,
             kv_heads=2, qk_scale=0.125, out=out, lse=torch.zeros(n, heads))
    wide = _aligned(n, 2 * heads * d)
    ints, floats = out.view(-1).view(torch.int32), out.view(-1).view(torch.float32)
    a.update({"query, shifted": dict(q=buf[:size].view(n, heads, d), out=buf[heads * d:size + heads * d].view(n, heads, d)),
              "query, strided": dict(q=wide[:, :heads * d].view(n, heads, d), out=wide.view(-1)[:size].view(n, heads, d)),
              "key": dict(k_cache=buf[:6 * 16 * 2 * d].view(6, 16, 2, d), out=buf[64:64 + size].view(n, heads, d)),
              "value": dict(v_cache=buf[:6 * 16 * 2 * d].view(6, 16, 2, d), out=buf[:size].view(n, heads, d)),
              "tables": dict(block_tables=ints[:12].view(3, 4)), "lengths": dict(seq_len=ints[4:7]),
              "lse": dict(lse=floats[:n * heads].view(n, heads)), "slopes": dict(mask_type=3, slopes=floats[16:16 + heads]),
              "lse on lengths": dict(lse=(x := torch.zeros(n, heads)), kv_seq_len=x.view(-1)[:3].view(torch.int32))}[which])
    with pytest.raises(ala.AlaError) as e:
        ala.plan_paged_attention(**a)
    assert e.value.status == 4, str(e.value)


def test_differential_attention_whose_output_shares_memory_is_refused():
    out = _aligned(10, 8, 64)
    a = dict(q=_aligned(10, 16, 32), k_cache=_aligned(6, 16, 4, 32), v_cache=_aligned(6, 16, 2, 64), block_tables=_i32(3, 4),
             seq_len=_i32(3), kv_seq_len=_i32(3), lam=torch.zeros(8), mask_type=9, heads=8, kv_heads=2, qk_scale=0.125, out=out)
    shared = out.view(-1).view(torch.float32)
    for over in (dict(lam=shared[:8]), dict(norm_weight=shared[8:72])):
        with pytest.raises(ala.AlaError) as e:
            ala.plan_paged_diff_attention(**{**a, **over})
        assert e.value.status == 4, str(e.value)


def test_attention_may_write_over_its_dense_query():
    q, cache = _aligned(10, 8, 64), _aligned(6, 16, 2, 64)
    assert ala.plan_paged_attention(q, cache, cache, _i32(3, 4), _i32(3), _i32(3), 9, 8, 2, 0.125, out=q)[1] is q
    q2 = _aligned(10, 16, 32)
    out = q2.view(10, 8, 64)
    ala.plan_paged_diff_attention(q2, cache.view(6, 16, 4, 32), cache, _i32(3, 4), _i32(3), _i32(3), torch.zeros(8), 9, 8, 2, 0.125, out=out)


# ---------------------------------------------------------------------------------------------- devices

def test_whether_a_stream_is_captured_is_asked_of_the_tensors_device(monkeypatch):
    # the current stream of the tensors' device, not of the device that happens to be current
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    bound, launched = [], []
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: index)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == 1)
    cache = _aligned(6, 16, 2, 64)
    for index, binds in ((1, False), (0, True)):
        op, _ = ala.plan_paged_attention(_aligned(3, 4, 64), cache, cache, _i32(3, 4), _i32(3), _i32(3), 9, 4, 2, 0.125)
        op._index = index
        op._execute = lambda *a: launched.append(current[0]) or 0
        monkeypatch.setattr(op, "bind", lambda stream: bound.append(index), raising=False)
        op()
        assert bound == ([index] if binds else []) and launched.pop() == index
        bound.clear()
        current[0] = 1 - current[0]
        op()
        assert bound == ([index] if binds else []) and launched.pop() == index
        bound.clear()
        current[0] = 0


# ---------------------------------------------------------------------------------------------- the remainder of P

def carried_bound(c, monkeypatch):
    """(out, bound of out) where P is multiplied as its rounding and the rounding of what that dropped: with u the half step of
    the type, the first is off by at most u p, and the second by u of that, so P by u^2 p; the output's rounding u |O| stays.
    Everything else is paged_ref's bound (fp16 weights that are subnormal lose up to 2^-25 either way)."""
    u = paged_ref.HALF[c["q"].dtype]
    with monkeypatch.context() as m:
        m.setattr(paged_ref, "HALF", {c["q"].dtype: u * u})
        out, _, tol, _ = paged_ref.attention(c)
    return out, tol + u * out.abs()


def _rounded_p(c, carry):
    """The output with P rounded as the kernels round it, all else in 64 bits; every sequence's keys in one page."""
    maps, group, dtype, at = c["maps"], c["heads"] // c["kv_heads"], c["q"].dtype, 0
    out = torch.zeros(int(c["seq"].sum()), c["heads"], c["v"].shape[-1], dtype=torch.float64)
    for b, (n, kv) in enumerate(zip(c["seq"].tolist(), c["kv"].tolist())):
        page = c["tables"][b, 0].long()
        k, v = c["k"][page, :kv].double(), c["v"][page, :kv].double()
        for h in range(c["heads"]):
            for m in range(maps):
                x = c["q"][at:at + n, h * maps + m].double() @ k[:, h // group * maps + m].T * c["scale"]
                p = torch.exp(x - x.amax(1, keepdim=True))
                hi = p.to(dtype).double()
                used = hi + (p - hi).to(dtype).double() if carry else hi
                w = 1.0 if m == 0 else -float(c["lam"][h])
                out[at:at + n, h] += w * (used @ v[:, h // group]) / p.sum(1, keepdim=True)
        at += n
    return out.to(dtype).double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("maps,d", [(1, 64), (2, 64), (1, 128), (2, 32)])
def test_the_bound_of_a_carried_remainder_notices_its_loss(maps, d, dtype, monkeypatch):
    c = paged_ref.make_case([(1, 20), (1, 33), (1, 60)], 8, 2, d, dtype, 64, 0, 5 + d, maps=maps)
    c["scale"] /= 16  # small scores: their own errors are below those of P
    ref, tol = carried_bound(c, monkeypatch)
    assert ((_rounded_p(c, True) - ref).abs() <= tol).all()
    lost = (_rounded_p(c, False) - ref).abs() > tol
    assert lost.float().mean() > 0.005
