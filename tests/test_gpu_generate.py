"""Generation over the paged cache against the training stack's attention over whole
sequences."""
import pytest
import torch
import torch.nn.functional as F

import partial_activation_sync_gb300 as caat
from partial_activation_sync_gb300.caatnet import CAATNet, rope_tables
from partial_activation_sync_gb300.generate import Generator

pytestmark = pytest.mark.gpu


def _model():
    torch.manual_seed(1)
    return CAATNet(vocab=1000, h=256, heads=16, layers=3, ffn=512, t=8, p=0.5, seq=128, std=0.06).cuda().bfloat16()


@torch.no_grad()
def _full_logits(m, tokens):
    """The training forward's logits [batch, seq, vocab]."""
    B, S = tokens.shape
    x = F.embedding(tokens.reshape(-1), m.emb).unsqueeze(0).expand(m.t, B * S, m.h).contiguous()
    cos, sin = rope_tables(S, m.h // m.heads, x.device, x.dtype)
    for blk in m.blocks:
        x = blk(x, cos, sin, B, S, m.sel())
    return (m.ln_f(x.mean(dim=0)) @ m.emb.t()).view(B, S, -1).float()


def _rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def test_logits_match_the_training_stack():
    # The cache rounds keys and values to e4m3, at most 2^-4 of each: attention outputs, and
    # with them the logits, stay within that of the training stack's.
    m = _model()
    tokens = torch.randint(0, 1000, (3, 40)).cuda()
    want = _full_logits(m, tokens)
    gen = Generator(m, 3, 64, page=16)
    got = gen.prefill([tokens[0, :37], tokens[1, :20], tokens[2, :1]])
    assert _rel(got, torch.stack([want[0, 36], want[1, 19], want[2, 0]])) < 2.0 ** -4
    # a further piece for two of them, then single tokens
    got = gen.prefill([tokens[0, 37:38], tokens[1, 20:33], tokens[2, 1:17]])
    assert _rel(got, torch.stack([want[0, 37], want[1, 32], want[2, 16]])) < 2.0 ** -4
    for i in range(2):
        got = gen.decode(torch.stack([tokens[0, 38 + i], tokens[1, 33 + i], tokens[2, 17 + i]]))
        assert _rel(got, torch.stack([want[0, 38 + i], want[1, 33 + i], want[2, 17 + i]])) < 2.0 ** -4
    assert caat.device_status() == 0


def test_generate_replays_what_single_steps_sample():
    m = _model()
    prompts = [torch.randint(0, 1000, (n,)).cuda() for n in (5, 33)]
    u = torch.rand(12, 2, device="cuda")
    gen = Generator(m, 2, 64, page=16)
    out = gen.generate(prompts, 12, u, temperature=0.9, top_k=40, top_p=0.9)
    gen.kv_len.zero_()
    again = gen.generate(prompts, 12, u, temperature=0.9, top_k=40, top_p=0.9)
    assert torch.equal(out, again)
    # the same by hand, without the graph
    one = Generator(m, 2, 64, page=16)
    how = [torch.full((2,), 0.9, device="cuda"), torch.full((2,), 40, dtype=torch.int32, device="cuda"),
           torch.full((2,), 0.9, device="cuda"), torch.zeros(2, device="cuda")]
    tok, _ = caat.sample_tokens(one.prefill(prompts), u[0].contiguous(), *how)
    assert torch.equal(tok, out[:, 0])
    for i in range(1, 12):
        tok, _ = caat.sample_tokens(one.decode(tok), u[i].contiguous(), *how)
        assert torch.equal(tok, out[:, i])
    # greedy: a temperature of 0 takes the largest logit
    gen.kv_len.zero_()
    greedy = gen.generate(prompts, 1, u, temperature=0.0)
    gen.kv_len.zero_()
    assert torch.equal(greedy[:, 0].long(), gen.prefill(prompts).float().argmax(-1))
    assert caat.device_status() == 0
