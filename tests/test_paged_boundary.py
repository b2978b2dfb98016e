"""Refusals of the paged serving operators (ala_paged_*): every one is made on the host, before any GPU work."""
import ctypes

import pytest
import torch

import paged_attention_varlen_b200 as ala


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


def _attn(**over):
    a = dict(q=_aligned(10, 8, 64), k_cache=_aligned(6, 16, 2, 64), v_cache=_aligned(6, 16, 2, 64), block_tables=_i32(3, 4),
             seq_len=_i32(3), kv_seq_len=_i32(3), mask_type=9, heads=8, kv_heads=2, qk_scale=0.125)
    a.update(over)
    return ala.plan_paged_attention(**a)


def _diff(**over):
    a = dict(q=_aligned(10, 16, 32), k_cache=_aligned(6, 16, 4, 32), v_cache=_aligned(6, 16, 2, 64), block_tables=_i32(3, 4),
             seq_len=_i32(3), kv_seq_len=_i32(3), lam=torch.zeros(8), mask_type=9, heads=8, kv_heads=2, qk_scale=0.125)
    a.update(over)
    return ala.plan_paged_diff_attention(**a)


def test_valid_plans_need_no_gpu():
    op, out = _attn()
    assert out.shape == (10, 8, 64) and op.workspace_size > 0
    op, out = _diff(norm_weight=torch.ones(64))
    assert out.shape == (10, 8, 64) and op.workspace_size > 0
    # the workspace depends on the head size alone: any number of tokens and sequences
    small, _ = _attn()
    big, _ = _attn(q=_aligned(1000, 8, 64), block_tables=_i32(300, 9), seq_len=_i32(300), kv_seq_len=_i32(300))
    assert small.workspace_size == big.workspace_size


def test_a_slice_of_a_fused_projection_is_taken_with_its_stride():
    fused = _aligned(10, 1024)
    op, out = _attn(q=fused[:, 512:].view(10, 8, 64))
    assert out.is_contiguous()
    with pytest.raises(ValueError):
        _attn(q=_aligned(10, 64, 8).transpose(1, 2))  # a token's row is not dense
    with pytest.raises(ValueError):
        _attn(q=_aligned(1, 8, 64).expand(10, 8, 64))  # every token the same memory


@pytest.mark.parametrize("over,status", [
    (dict(mask_type=1), 4), (dict(heads=0), 4), (dict(heads=7), 4), (dict(kv_heads=3), 4), (dict(kv_heads=0), 4),
    (dict(qk_scale=float("nan")), 4), (dict(qk_scale=float("inf")), 4),
    (dict(q=torch.zeros(10, 8, 64)), 3),                                           # fp32
    (dict(v_cache=_aligned(6, 16, 2, 64, dtype=torch.float16)), 3),
    (dict(k_cache=_aligned(6, 16, 4, 64)), 2), (dict(v_cache=_aligned(7, 16, 2, 64)), 2),
    (dict(k_cache=_aligned(6, 8, 2, 64), v_cache=_aligned(6, 8, 2, 64)), 5),       # blockSize % 16
    (dict(k_cache=_aligned(0, 16, 2, 64), v_cache=_aligned(0, 16, 2, 64)), 2),     # no blocks
    (dict(q=_aligned(10, 8, 60), k_cache=_aligned(6, 16, 2, 60), v_cache=_aligned(6, 16, 2, 60)), 5),
    (dict(q=_aligned(10, 8, 264), k_cache=_aligned(6, 16, 2, 264), v_cache=_aligned(6, 16, 2, 264)), 5),
    (dict(q=_aligned(2, 258, 8), k_cache=_aligned(6, 16, 2, 8), v_cache=_aligned(6, 16, 2, 8), heads=258), 5),
    (dict(seq_len=_i32(2)), 2), (dict(kv_seq_len=_i32(3, 1)), 2), (dict(seq_len=torch.zeros(3)), 3),
    (dict(block_tables=_i32(4)), 2),
    (dict(mask_type=3), 1), (dict(slopes=torch.ones(8)), 4), (dict(mask_type=3, slopes=torch.ones(7)), 2),
    (dict(mask_type=4, slopes=torch.ones(8), q=_aligned(10, 8, 136), k_cache=_aligned(6, 16, 2, 136),
          v_cache=_aligned(6, 16, 2, 136)), 4),
    (dict(lse=torch.zeros(10)), 2), (dict(lse=torch.zeros(9, 8)), 2), (dict(lse=_aligned(10, 8)), 3),
    (dict(out=_aligned(10, 8, 32)), 2), (dict(out=_aligned(11 * 512)[8:8 + 5120].view(10, 8, 64)), 4),  # 16-byte aligned only
])
def test_attention_refuses(over, status):
    with pytest.raises(ala.AlaError) as e:
        _attn(**over)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("over,status", [
    (dict(mask_type=3), 4), (dict(heads=3), 4), (dict(lam=torch.zeros(16)), 2), (dict(lam=_aligned(8)), 3),
    (dict(norm_weight=torch.ones(32)), 2), (dict(norm_eps=-1.0), 4), (dict(out_scale=float("inf")), 4),
    (dict(v_cache=_aligned(6, 16, 4, 32)), 2), (dict(k_cache=_aligned(6, 16, 2, 64)), 2),
    (dict(q=_aligned(10, 16, 136), k_cache=_aligned(6, 16, 4, 136), v_cache=_aligned(6, 16, 2, 272)), 5),
    (dict(q=_aligned(10, 260, 8), k_cache=_aligned(6, 16, 4, 8), v_cache=_aligned(6, 16, 2, 16), heads=130,
          lam=torch.zeros(130)), 5),
])
def test_diff_attention_refuses(over, status):
    with pytest.raises(ala.AlaError) as e:
        _diff(**over)
    assert e.value.status == status, str(e.value)


def test_executions_refuse_a_foreign_op_and_a_bad_workspace():
    op, _ = _attn()
    L, fake = ala.lib(), 1 << 20
    assert L.ala_paged_diff_attention(fake, op.workspace_size, op._handle, None) == 4
    assert L.ala_paged_attention(fake, op.workspace_size, None, None) == 1
    assert L.ala_paged_attention(None, op.workspace_size, op._handle, None) == 1
    assert L.ala_paged_attention(fake, op.workspace_size - 1, op._handle, None) == 6
    assert L.ala_paged_attention(fake + 16, op.workspace_size, op._handle, None) == 4
    assert L.ala_op_bind_workspace(op._handle, fake + 16, op.workspace_size, None) == 4
    assert L.ala_op_bind_workspace(op._handle, None, 0, None) == 0


def _step_args(**over):
    a = dict(seqLen=_i32(3), contextLens=_i32(3), finished=_i32(3), blockTables=_i32(3, 4), freeBlocks=_i32(20),
             freeCount=_i32(1), blockSize=16, kvSeqLen=_i32(3), freeCountOut=_i32(1), cuSeqLen=_i32(4),
             slotMapping=_i32(12), positions=_i32(12), status=_i32(1))
    a.update(over)
    return a


def _step(**over):
    a = _step_args(**over)
    ts = {k: x if isinstance(x, int) else ala.tensor(x) for k, x in a.items()}
    return ala.lib().ala_paged_step(*[x if isinstance(x, int) or x is None else ctypes.byref(x) for x in ts.values()], None)


_shared = _i32(40)


@pytest.mark.parametrize("over,status", [
    (dict(seqLen=None), 1), (dict(status=None), 1), (dict(seqLen=torch.zeros(3)), 3), (dict(blockSize=0), 4),
    (dict(blockTables=_i32(3)), 2), (dict(contextLens=_i32(4)), 2), (dict(finished=_i32(2)), 2), (dict(cuSeqLen=_i32(3)), 2),
    (dict(freeCount=_i32(2)), 2), (dict(positions=_i32(11)), 2), (dict(freeBlocks=_i32(4, 5)), 2),
    (dict(blockSize=1 << 29), 5),
    (dict(seqLen=_shared[:3], kvSeqLen=_shared[:3]), 4), (dict(contextLens=_shared[:3], kvSeqLen=_shared[1:4]), 4),
    (dict(slotMapping=_shared[:12], positions=_shared[6:18]), 4), (dict(freeCount=_shared[:1], status=_shared[:1]), 4),
    (dict(freeBlocks=_shared[:20], freeCount=_shared[19:20]), 4),
    (dict(seqLen=_i32(8193), contextLens=_i32(8193), finished=None, blockTables=_i32(8193, 1), kvSeqLen=_i32(8193),
          cuSeqLen=_i32(8194)), 5),
])
def test_step_refuses(over, status):
    assert _step(**over) == status, ala.lib().ala_last_error().decode()


_kv = torch.zeros(4, 2, 24)


@pytest.mark.parametrize("over", [
    dict(key=None), dict(slots=torch.zeros(4)), dict(slots=_i32(5)), dict(slots=_i32(4, 1)), dict(value=None),
    dict(key_cache=torch.zeros(3, 16, 2, 32)), dict(key_cache=torch.zeros(3, 16, 2, 24, dtype=torch.float16)),
    dict(value_cache=torch.zeros(3, 32, 2, 24)), dict(key_cache=torch.zeros(48, 48)), dict(key_stride=47),
    dict(key_stride=-1)])
def test_write_refuses(over):
    a = dict(key=_kv, key_stride=0, value=_kv, value_stride=0, slots=_i32(4), key_cache=torch.zeros(3, 16, 2, 24),
             value_cache=torch.zeros(3, 16, 48))
    a.update(over)
    ts = [x if isinstance(x, int) else ala.tensor(x) for x in a.values()]
    st = ala.lib().ala_paged_write(*[x if isinstance(x, int) or x is None else ctypes.byref(x) for x in ts], None)
    assert st in (1, 2, 3, 4), ala.lib().ala_last_error().decode()


def test_python_refuses_tensors_on_different_devices():
    meta = torch.zeros(3, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError):
        _attn(seq_len=meta)
    with pytest.raises(ValueError):
        ala.plan_paged_write(_kv, _kv, _i32(4), torch.zeros(3, 16, 48), torch.zeros(3, 16, 48, device="meta"))


def _odd(shape, dtype):
    """A tensor whose address is one byte off its elements' alignment."""
    t = ala.AlaTensor()
    buf = (ctypes.c_uint8 * 4096)()
    t.data = (ctypes.addressof(buf) // 8 + 1) * 8 + 1
    t.dtype, t.ndim = dtype, len(shape)
    for i, s in enumerate(shape):
        t.dims[i] = s
    t._buf = buf
    return t


@pytest.mark.parametrize("name,shape", [("seqLen", (3,)), ("blockTables", (3, 4)), ("status", (1,)), ("slotMapping", (12,))])
def test_step_refuses_an_address_off_its_elements(name, shape):
    ts = {k: x if isinstance(x, int) else ala.tensor(x) for k, x in _step_args().items()}
    ts[name] = _odd(shape, ala.I32)
    assert ala.lib().ala_paged_step(*[x if isinstance(x, int) else ctypes.byref(x) for x in ts.values()], None) == 4


@pytest.mark.parametrize("which", ["tables", "seq", "kv", "lse", "slots"])
def test_attention_and_write_refuse_an_address_off_its_elements(which):
    L = ala.lib()
    if which == "slots":
        ts = [ala.tensor(_kv), ala.tensor(_kv), _odd((4,), ala.I32), ala.tensor(torch.zeros(3, 16, 2, 24)), ala.tensor(torch.zeros(3, 16, 48))]
        r = [ctypes.byref(t) for t in ts]
        assert L.ala_paged_write(r[0], 0, r[1], 0, r[2], r[3], r[4], None) == 4
        return
    q, k, v, out = _aligned(10, 8, 64), _aligned(6, 16, 2, 64), _aligned(6, 16, 2, 64), _aligned(10, 8, 64)
    ts = dict(tables=ala.tensor(_i32(3, 4)), seq=ala.tensor(_i32(3)), kv=ala.tensor(_i32(3)), lse=ala.tensor(torch.zeros(10, 8)))
    ts[which] = _odd({"tables": (3, 4), "lse": (10, 8)}.get(which, (3,)), ala.F32 if which == "lse" else ala.I32)
    tq, tk, tv, to = (ala.tensor(x) for x in (q, k, v, out))
    ws, h = ctypes.c_uint64(0), ctypes.c_void_p(0)
    b = ctypes.byref
    st = L.ala_paged_attention_get_workspace_size(b(tq), 0, b(tk), b(tv), b(ts["tables"]), b(ts["seq"]), b(ts["kv"]), None, 9, 8, 2, 0.1,
                                                  b(to), b(ts["lse"]), b(ws), b(h))
    assert st == 4 and not h.value
