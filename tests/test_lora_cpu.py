"""lora_gemm without a GPU: refusals of the C call and of the binding.  Pointers are fake and never
dereferenced."""
import numpy as np
import pytest

import lora_ref
import quantized_sparse_moe_amd as q

A = 0x7F0000000000
S = 1 << 36                        # tensors far apart


def call(**kw):
    a = dict(a=A, b=A + S, scales=None, ranks=None, n=4, R=16, K=64, N=80, ids=A + 2 * S, x=A + 3 * S, T=5, ldx=64,
             base=A + 4 * S, ldb=80, y=A + 5 * S, dt=q.MOE_BF16, ldy=80, ws=A + 6 * S, wb=1 << 30)
    a.update(kw)
    return q.lib().lora_gemm(a["a"], a["b"], a["scales"], a["ranks"], a["n"], a["R"], a["K"], a["N"], a["ids"], a["x"], a["T"],
                             a["ldx"], a["base"], a["ldb"], a["y"], a["dt"], a["ldy"], a["ws"], a["wb"], None)


INVALID = [dict(T=-1), dict(N=-1), dict(n=-1), dict(dt=q.MOE_F16), dict(a=None), dict(a=A + 8), dict(b=None), dict(b=A + S + 2),
           dict(ids=None), dict(ids=A + 2 * S + 2), dict(x=None), dict(x=A + 3 * S + 2), dict(ldx=56), dict(ldx=68),
           dict(scales=A + 7 * S + 2), dict(ranks=A + 7 * S + 1), dict(y=None), dict(y=A + 5 * S + 1), dict(ldy=79),
           dict(base=A + 4 * S + 1), dict(ldb=79), dict(dt=q.MOE_F32, y=A + 5 * S + 2), dict(y=A + 4 * S, ldy=88),
           dict(y=A + 4 * S + 2), dict(y=A + 3 * S), dict(y=A), dict(y=A + S + 64), dict(y=A + 2 * S), dict(y=A + 6 * S),
           dict(scales=A + 5 * S + 4), dict(ranks=A + 5 * S + 4), dict(x=A + 6 * S), dict(base=A + 6 * S + 256), dict(ids=A + 6 * S)]
UNSUPPORTED = [dict(R=4), dict(R=12), dict(R=264), dict(R=0), dict(K=4), dict(K=68), dict(K=65544), dict(N=(1 << 23) + 1),
               dict(n=0), dict(n=65537), dict(T=(1 << 20) + 1)]


@pytest.mark.parametrize("i", range(len(INVALID)))
def test_invalid(i):
    assert call(**INVALID[i]) == q.MOE_ERR_INVALID, INVALID[i]


def test_limits_workspace_and_nothing_to_do():
    for kw in UNSUPPORTED:
        assert call(**kw) == q.MOE_ERR_UNSUPPORTED, kw
    need = q.lib().lora_workspace_size(5, 16)
    assert need >= 5 * 16 * 6
    for kw in (dict(ws=None), dict(ws=A + 6 * S + 64), dict(wb=need - 1)):
        assert call(**kw) == q.MOE_ERR_WORKSPACE, kw
    assert call(T=0, x=None, y=None, ws=None) == q.MOE_OK
    assert call(N=0, y=None, ws=None) == q.MOE_OK
    big = 2 ** 64 - 1
    assert q.lib().lora_workspace_size(5, 12) == big and q.lib().lora_workspace_size((1 << 20) + 1, 16) == big
    assert q.lib().lora_workspace_size(0, 16) == 0
    sizes = [q.lora_workspace_size(T, 64) for T in (1, 2, 100, 4096)]
    assert sizes == sorted(sizes)
    with pytest.raises(q.QsmoeError):
        q.lora_workspace_size(5, 12)


@pytest.mark.parametrize("kw", [dict(a=A + 6 * S), dict(b=A + 6 * S + 256), dict(scales=A + 6 * S), dict(ranks=A + 6 * S + 4),
                                dict(a=A + 6 * S - 4 * 16 * 64 * 2 + 16), dict(b=A + 6 * S - 4 * 80 * 16 * 2 + 16)])
def test_a_workspace_over_the_adapters_is_refused(kw):
    assert call(**kw) == q.MOE_ERR_INVALID


def test_binding_checks_its_arguments():
    import torch
    a, b = torch.zeros(3, 8, 16, dtype=torch.bfloat16), torch.zeros(3, 24, 8, dtype=torch.bfloat16)
    for bad in ((a[:, :4].contiguous(), b[:, :, :4].contiguous()), (a[:, :, :4].contiguous(), b), (a.float(), b), (a, b[:2]), (a, b[:, :, :4].contiguous()), (a[0], b), (a[:, :, ::2], b)):
        with pytest.raises(q.QsmoeError):
            q.LoraAdapters(*bad)
    for kw in (dict(scales=torch.ones(2)), dict(scales=torch.ones(3).half()), dict(ranks=torch.ones(3)),
               dict(ranks=torch.ones(6, dtype=torch.int32)[::2])):
        with pytest.raises(q.QsmoeError):
            q.LoraAdapters(a, b, **kw)
    ad = q.LoraAdapters(a, b)
    x, ids = torch.zeros(5, 16, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    for args, kw in (((ad, ids.long(), x), {}), ((ad, ids[:4], x), {}), ((ad, ids, x.float()), {}), ((ad, ids, x[:, :8]), {}),
                     ((ad, ids, x), dict(y=torch.zeros(5, 23))), ((ad, ids, x), dict(base=torch.zeros(4, 24))),
                     ((ad, ids, x), dict(base=torch.zeros(5, 24), y_dtype=torch.bfloat16)), ((ad, ids, x), {})):
        with pytest.raises(q.QsmoeError):                    # (the last: tensors on the host)
            q.lora_gemm(*args, **kw)
    with pytest.raises(q.QsmoeError):
        q.mx4_gemm(None, None, 25, 16, x, adapters=ad, adapter_ids=ids)
    with pytest.raises(q.QsmoeError):
        q.mx4_gemm(None, None, 24, 16, x, adapters=ad)
    with pytest.raises(q.QsmoeError):                        # (before the product is enqueued)
        q.mx4_gemm(None, None, 24, 16, x, adapters=ad, adapter_ids=ids, adapter_workspace=torch.zeros(8, dtype=torch.uint8))


def test_adapters_are_checked_before_a_product_is_enqueued(monkeypatch):
    """mx4_gemm(adapters=): whatever lora_gemm refuses, y is not written first.  (Host tensors, taken as if
    they were on a GPU but in the first case; every call is refused.)"""
    import torch
    enqueued = []
    monkeypatch.setattr(q, "_mx4_product", lambda *a: enqueued.append(a))
    bf = torch.bfloat16
    a, b = torch.zeros(3, 8, 32, dtype=bf), torch.zeros(3, 24, 8, dtype=bf)
    x, ids = torch.zeros(5, 32, dtype=bf), torch.zeros(5, dtype=torch.int32)
    buf = torch.zeros(1 << 14, dtype=torch.uint8)
    buf = buf[-buf.data_ptr() % 256:]
    ws = buf[:8192]

    def refused(ad=q.LoraAdapters(a, b), N=24, ids=ids, y=None, ws=ws, **kw):
        with pytest.raises(q.QsmoeError):
            q.mx4_gemm(None, None, N, 32, x, y=y, adapters=ad, adapter_ids=ids, adapter_workspace=ws, **kw)
        assert not enqueued

    refused()                                                # another device
    monkeypatch.setattr(q, "_mx4_stream", lambda *a: (0, True))
    many = q.LoraAdapters(torch.zeros(65537, 8, 8, dtype=bf), torch.zeros(65537, 1, 8, dtype=bf))
    with pytest.raises(q.QsmoeError):
        q.mx4_gemm(None, None, 1, 8, x[:, :8].contiguous(), adapters=many, adapter_ids=ids, adapter_workspace=ws)
    refused(q.LoraAdapters(torch.zeros(3 * 8 * 32 + 1, dtype=bf)[1:].view(3, 8, 32), b))     # not aligned
    over = ws.view(torch.float32)
    refused(y=over[:120].view(5, 24))                        # y over the workspace
    refused(ids=ws.view(torch.int32)[:5])
    refused(y=b.view(-1)[:120].view(5, 24))                  # and over an adapter
    refused(y_dtype=torch.float16)
    refused(ws=buf[:64])
    refused(ws=buf[64:8256])
    assert not enqueued


def test_adapter_ids_without_adapters_are_refused(monkeypatch):
    import torch
    monkeypatch.setattr(q, "_mx4_product", lambda *a: pytest.fail("enqueued"))
    with pytest.raises(q.QsmoeError):
        q.mx4_gemm(None, None, 24, 32, torch.zeros(5, 32, dtype=torch.bfloat16), adapter_ids=torch.zeros(5, dtype=torch.int32))


def test_reference_by_hand():
    a = np.array([[[1.0, 0.0], [0.0, 2.0]], [[1.0, 1.0], [0.0, 0.0]]])
    b = np.array([[[1.0, 1.0]], [[3.0, np.nan]]])
    y, bound = lora_ref.forward(a, b, [0, 1, -1, 2], np.array([[1.0, 2.0]] * 4), np.full((4, 1), 10.0), scales=[1.0, 0.5],
                                ranks=[2, 1])
    assert y[:, 0].tolist() == [15.0, 14.5, 10.0, 10.0] and (bound < 1e-3).all()
