"""The attention half and the expert-slot cache together: a small decoder whose
decode steps agree with one pass over the whole texts, also after its sequences
were forked, rolled back and compacted."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def rows(*s):
    return torch.tensor(s, dtype=torch.int32, device="cuda")


@pytest.fixture(params=[torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def decoder(request):
    from examples.decoder import Decoder
    d = Decoder(dtype=request.param)
    yield d
    d.close()


def tolerance(d):
    # logits are sums of 64 products of order one; f32 rounds about 1e-6 a layer, bf16 2^-8 of a
    # hidden state at some ten places, over sqrt(64) = 8 times their size
    return 1e-3 if d.dtype == torch.float32 else 8 * 10 * 2.0 ** -8


def test_decode_steps_agree_with_one_pass(decoder):
    d = decoder
    prompts = [[5, 17, 3, 88, 41], [9] * 33, [1]]
    logits = d.prompt(prompts, [0, 1, 2])
    text = [list(p) for p in prompts]
    for i in range(18):
        token = [(11 * i + 7 * j) % 97 for j in range(3)]
        for t, x in zip(text, token):
            t.append(x)
        logits = d.step(token, [0, 1, 2])
    again = d.prompt(text, [3, 4, 5])
    d.kv.check()
    assert torch.isfinite(logits).all()
    assert float((logits - again).abs().max()) <= tolerance(d)


def test_forked_rolled_back_and_compacted_sequences(decoder):
    d = decoder
    prompt = [3, 14, 15, 92, 65, 35, 89, 79, 32, 38, 46, 26, 43, 38, 32, 79, 50, 28, 84, 19]
    d.prompt([prompt, [8] * 40], [0, 1])
    d.kv.fork(rows(0, 0), rows(2, 3))                       # two continuations of the first prompt
    d.step([7, 8], [2, 3])
    d.kv.free(rows(1))                                      # the second one ends; its pages close up
    d.kv.compact()
    a = d.step([70, 80], [2, 3])
    d.kv.truncate(rows(3), torch.tensor([len(prompt) + 1], dtype=torch.int32, device="cuda"))
    b = d.step([81, 1], [3, 0])                             # another token instead, and one for the parent
    texts = [prompt + [7, 70], prompt + [8, 80], prompt + [8, 81], prompt + [1]]
    want = d.prompt(texts, [4, 5, 6, 7])
    d.kv.check()
    got = torch.stack([a[0], a[1], b[0], b[1]])
    assert float((got - want).abs().max()) <= tolerance(d)
    held = d.kv.refs.clone()
    d.kv.free(rows(0, 2, 3, 4, 5, 6, 7))
    d.kv.check()
    assert int(held.sum()) > 0 and not d.kv.refs.any() and not d.kv.lens.any() and (d.kv.table == -1).all()
