"""PagedCache and pack_latents refuse tensors that their kernels would read or write out of
range: a batch that is not padded to max_tokens, another type, a view."""
import pytest
import torch

from long_context_sparse_04_b200 import workload as W


def test_argument_check():
    x = torch.zeros(4, 6)
    cpu = torch.device("cpu")
    assert W._tensor(x, "x", (4, 6), (torch.float32,), cpu).value == x.data_ptr()
    assert W._tensor(x, "x", (4, 6), (torch.uint8, torch.float32), cpu).value == x.data_ptr()
    for bad in (x[:3], x.double(), x.t().contiguous(), x.t(), torch.zeros(6, 4).t(), torch.zeros(4, 12)[:, ::2], x.to("meta")):
        with pytest.raises(ValueError, match="^x: contiguous torch.float32 of shape"):
            W._tensor(bad, "x", (4, 6), (torch.float32,), cpu)


@pytest.mark.gpu
def test_paged_cache_refuses():
    B, M, topk = 2, 8, 16
    pl = W.DevicePlanner(num_seqs=B, page_size=64, num_pages=8, max_pages_per_seq=4, max_tokens=M)
    ca = W.PagedCache(pl, topk=topk)
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    new = dict(k_new=z(M, 128), latent_new=z(M, 576, dtype=bf))
    step = dict(q_idx=z(M, 64, 128, dtype=torch.uint8), q_scale=z(M, 64), w=z(M, 64), q=z(M, 128, 576, dtype=bf),
                out=z(M, 128, 512, dtype=bf), lse=z(M, 128))
    get = dict(slot=z(5, dtype=torch.int64), k_out=z(5, 128), latent_out=z(5, 576, dtype=bf))
    pl.n_new.fill_(1)
    pl.plan()
    ca.append(**new), ca.decode_step(**step), ca.read(**get)
    ca.decode_step(**dict(step, lse=None, q_idx=step["q_idx"].view(torch.float8_e4m3fn)))
    ca.read(get["slot"], latent_out=get["latent_out"])
    for call, args in ((ca.append, new), (ca.decode_step, step), (ca.read, get)):
        for name, x in args.items():
            bad = [x.cpu(), x.to(torch.int16), torch.stack([x, x], dim=-1)[..., 0]]
            if name != "slot":
                bad += [x[:-1], x.repeat(2, *[1] * (x.dim() - 1))]
            for y in bad:
                with pytest.raises(ValueError, match=f"^{name}: contiguous"):
                    call(**dict(args, **{name: y}))
    assert pl.status() == (0, -1) and ca.status() == (0, -1)


@pytest.mark.gpu
def test_pack_latents():
    pl = W.DevicePlanner(num_seqs=1, page_size=64, num_pages=2, max_pages_per_seq=2, max_tokens=1)
    d = W.PagedCache(pl, topk=16).dims
    x = torch.randn(7, 576, device="cuda").bfloat16()
    assert W.pack_latents(d, x).shape == (7, 416) and W.pack_latents(d, x[:0]).shape == (0, 416)
    for bad in (x.float(), x[:, :575], torch.randn(576, 7, device="cuda").bfloat16().t(), x.cpu()):
        with pytest.raises(ValueError, match="^latent"):
            W.pack_latents(d, bad)
    x[3, 511] = float("inf")
    with pytest.raises(ValueError, match="row 3 has an infinity"):
        W.pack_latents(d, x)
