"""The calls of a replica's step together, as they would be used: embedding, an attention block
with the norm and rotation of queries and keys, distillation into the tied output layer, all
gradients, their global norm, and the clipped gradients in the replica's slab, against
autograd in 64 bits; then the ZeRO-1 step on the slabs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

V, D, HD, Hq, Hk, K = 300, 128, 32, 4, 2, 8
SEQS = [50, 1, 70]
T = sum(SEQS)


def forward64(p, ids, pos, f, t_ids, t_logits):
    h = p["E"][ids] * D ** 0.5
    qkv = (h @ p["W"]).view(T, Hq + 2 * Hk, HD)
    q, k, v = qkv.split([Hq, Hk, Hk], dim=1)
    a = pos.double()[:, None] * f.double()
    c, s = a.cos()[:, None], a.sin()[:, None]

    def rope(x, w):
        x = x * (x.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        u, z = x.chunk(2, dim=-1)
        return torch.cat([u * c - z * s, z * c + u * s], -1)
    q, k = rope(q, p["wq"]), rope(k, p["wk"])
    outs, at = [], 0
    for n in SEQS:
        r = slice(at, at + n)
        z = torch.einsum("qhd,khd->hqk", q[r], k[r].repeat_interleave(Hq // Hk, 1)) * HD ** -0.5
        z = z.masked_fill(~torch.ones(n, n, dtype=torch.bool, device=z.device).tril(), -torch.inf)
        outs.append(torch.einsum("hqk,khd->qhd", z.softmax(-1), v[r].repeat_interleave(Hq // Hk, 1)))
        at += n
    y = h + torch.cat(outs).reshape(T, Hq * HD) @ p["O"]
    logp = torch.log_softmax((y / D) @ p["E"].T, 1)
    lq = torch.log_softmax(t_logits.double(), 1)
    return (lq.exp() * (lq - logp.gather(1, t_ids))).sum(1)


def step(dpz, p, ids, pos, f, t_ids, t_logits, dt):
    """Loss and gradients by the library's calls, with products of torch between them."""
    new = lambda *s, t=dt: torch.empty(*s, dtype=t, device="cuda")       # noqa: E731
    cu = torch.tensor([0, 50, 51, 121], dtype=torch.int32, device="cuda")
    h, qkv, n = new(T, D), new(T, (Hq + 2 * Hk) * HD), new(T, Hq + 2 * Hk, HD)
    dpz.lm_embedding(p["E"], ids, h, scale=D ** 0.5)
    torch.matmul(h, p["W"], out=qkv)
    heads = lambda x: x.view(T, Hq + 2 * Hk, HD).split([Hq, Hk, Hk], dim=1)  # noqa: E731
    q, k, v = heads(qkv)
    nq, nk, _ = heads(n)
    rope = dict(wq=p["wq"], wk=p["wk"], positions=pos, inv_freq=f)
    dpz.attn_qk_norm_rope(q, k, nq, nk, **rope)
    o, lse = new(T, Hq, HD), new(Hq, T, t=torch.float32)
    kw = dict(causal=True, cu_q=cu, cu_k=cu)
    dpz.attn_forward(nq, nk, v, o, lse=lse, **kw)
    y = torch.addmm(h, o.view(T, Hq * HD), p["O"])
    logits, loss = new(T, V), new(T, t=torch.float32)
    torch.matmul(y / D, p["E"].T, out=logits)
    w = torch.full((T,), 1.0 / T, device="cuda")
    dpz.lm_distill_step(logits, t_ids, t_logits, w, loss, logits)
    g = {m: torch.empty_like(x) for m, x in p.items()}
    torch.matmul(logits.T, y / D, out=g["E"])
    dy = (logits @ p["E"]) / D
    torch.matmul(o.view(T, -1).T, dy, out=g["O"])
    do = (dy @ p["O"].T).view(T, Hq, HD)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = heads(dqkv)
    dpz.attn_grad(nq, nk, v, o, lse, do, dq, dk, dv, dpz.attn_grad_workspace(T, T, 3, Hq, Hk, HD), **kw)
    dpz.attn_qk_norm_rope_grad(q, k, dq, dk, dq, dk, dpz.attn_qk_norm_rope_workspace(T, Hq, Hk, HD),
                               dwq=g["wq"], dwk=g["wk"], **rope)
    torch.matmul(h.T, dqkv, out=g["W"])
    dh = dy + dqkv @ p["W"].T
    dpz.lm_embedding_grad(dh, ids, g["E"], dpz.lm_embedding_workspace(T, V, D), base=g["E"],
                          scale=D ** 0.5)
    return loss, g


@pytest.mark.parametrize("dt,rel", [(torch.float32, 2e-5), (torch.bfloat16, 4e-2)])
def test_step_against_autograd(dt, rel):
    """rel: of each gradient's norm.  In fp32 each of a dozen steps in turn is within some 100 u
    (6e-6) of its terms; in bf16 about a dozen roundings of 2^-8, half of them at random,
    lie between the loss and the first layer's gradients."""
    import gradient_reduction_zero_gb300.dpz as dpz
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")        # noqa: E731
    p = dict(E=rand(V, D) * 0.5, W=rand(D, (Hq + 2 * Hk) * HD) * D ** -0.5 * 0.2,
             O=rand(Hq * HD, D) * (Hq * HD) ** -0.5, wq=1 + 0.2 * rand(HD), wk=1 + 0.2 * rand(HD))
    p = {n: x.to(dt) for n, x in p.items()}
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    pos = torch.cat([torch.arange(n, device="cuda") for n in SEQS])
    f = (10000.0 ** (-torch.arange(HD // 2, device="cuda") / (HD / 2))).float()
    t_logits, t_ids = torch.topk(rand(T, V) * 2, K, dim=1)
    loss, got = step(dpz, p, ids, pos, f, t_ids, t_logits, dt)
    p64 = {n: x.double().requires_grad_() for n, x in p.items()}
    want = forward64(p64, ids, pos, f, t_ids, t_logits)
    want.mean().backward()
    want = want.detach()
    assert float((loss.double() - want).norm() / want.norm()) <= rel
    for n in p:
        d = float((got[n].double() - p64[n].grad).norm() / p64[n].grad.norm())
        assert d <= rel, (n, d)

    # the global norm, and the clipped gradients in the slabs of two replicas
    names = sorted(p)
    lst = dpz.TensorList(got[n] for n in names)
    norm = torch.empty(1, device="cuda")
    dpz.tensors_norm(lst, norm, dpz.tensors_workspace(lst))
    total = torch.cat([got[n].double().view(-1) for n in names]).norm()
    assert abs(float(norm) - float(total)) <= 1e-6 * float(total)
    P = -(-sum(x.numel() for x in p.values()) // 16) * 16
    grads = torch.zeros(2, P, dtype=torch.bfloat16, device="cuda")
    clip = 0.5 * float(total)
    for r in range(2):
        views, at = [], 0
        for n in names:
            views.append(grads[r, at:at + p[n].numel()].view(p[n].shape))
            at += p[n].numel()
        dpz.tensors_clip(lst, norm, clip, out=dpz.TensorList(views))
        for n, x in zip(names, views):
            assert torch.equal(x, (got[n].float() * (clip / norm)).bfloat16()), n
    master, m, v = (torch.zeros(P, device="cuda") for _ in range(3))
    weights = torch.zeros(2, P, dtype=torch.bfloat16, device="cuda")
    ws = dpz.workspace(P, 2)
    cfg = dpz.make_cfg(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=1)
    dpz.dp_zero1_step(grads.view(-1), master, m, v, weights.view(-1), 2, cfg, ws=ws, norm_out=norm)
    avg = grads[0].double()                       # both replicas have the same gradients
    assert abs(float(norm) - float(avg.norm())) <= 1e-6 * float(avg.norm())
    assert torch.equal(weights[0], weights[1]) and bool((master != 0).any())
    assert dpz.device_status() == 0
