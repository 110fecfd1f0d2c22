"""The serving head under the C names, which take their sizes and strides from the tensors, against the functions that
make their outputs: the same bits."""
import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,N,K", [(1, 1025, 512), (7, 300, 129), (140, 700, 1000)])
def test_same_bits(n, N, K, dtype):
    dev, g = torch.device("cuda", 0), torch.Generator().manual_seed(n)
    w = torch.randint(-127, 128, (N, K + 3), generator=g).to(torch.int8).to(dev)[:, 1:K + 1]
    sw = (torch.rand((N,), generator=g) * 1e-3).to(dev)
    x = (torch.randn((n, K + 5), generator=g) * 2).to(DT[dtype]).to(dev)[:, 2:K + 2]
    gain = (1 + 0.1 * torch.randn((K,), generator=g)).to(dev)
    bytes_ = lambda count: torch.empty(count, dtype=torch.uint8, device=dev)  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device=dev)

    p = pkg.pack_i8(w, sw)
    packed = bytes_(pkg.packed_i8_bytes(N, K))
    assert pkg.ds_pack_i8(w, packed) == 0 and torch.equal(packed, p.packed)

    want_q, want_s = pkg.quantize_rows(x, gain=gain, eps=1e-5)
    q, s = torch.empty((n, K), dtype=torch.int8, device=dev), torch.empty(n, device=dev)
    assert pkg.ds_quantize_rows(x, q, s, gain=gain, eps=1e-5) == 0
    assert torch.equal(q, want_q) and torch.equal(s, want_s)

    want = pkg.linear_i8(q, s, p, dtype=DT[dtype])
    out = torch.full((n, N + 2), 5.0, dtype=DT[dtype], device=dev)
    ws = bytes_(pkg.linear_i8_workspace(n, N, K))
    assert pkg.ds_linear_i8(q, s, packed, sw, out[:, :N], N, K, workspace=ws, d_status=st, ldo=N + 2) == 0
    assert torch.equal(out[:, :N], want) and bool((out[:, N:] == 5.0).all())

    logits = torch.empty((n, N), dtype=DT[dtype], device=dev)
    ws = bytes_(pkg.head_i8_workspace(n, N, K))
    assert pkg.ds_head_i8(x, packed, sw, logits, ws, N, gain=gain, eps=1e-5, d_status=st) == 0
    assert torch.equal(logits, want)

    tau, u = torch.full((n,), 0.8, device=dev), torch.rand((n,), generator=g).to(dev)
    k = torch.full((n,), 40, dtype=torch.int32, device=dev)
    top_p, min_p = torch.full((n,), 0.9, device=dev), torch.full((n,), 0.01, device=dev)
    want_tok, want_lp = pkg.sample_filtered(out[:, :N], tau, u, top_k=k, top_p=top_p, min_p=min_p)
    tok, lp = torch.empty(n, dtype=torch.int32, device=dev), torch.empty(n, device=dev)
    assert pkg.ds_sample_filtered(out[:, :N], tau, u, tok, lp, top_k=k, top_p=top_p, min_p=min_p, d_status=st,
                                  ld=N + 2) == 0
    assert torch.equal(tok, want_tok) and torch.equal(lp, want_lp)
    assert int(st.item()) == 0

    with pytest.raises(pkg.DsError):
        pkg.ds_linear_i8(q, s, packed, sw, out, N, K, workspace=ws[:64])
    with pytest.raises(TypeError):
        pkg.ds_quantize_rows(x.half(), q, s)
