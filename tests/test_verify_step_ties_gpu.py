"""The verify step of examples/verify_step.py where logits tie."""
import pytest

torch = pytest.importorskip("torch")
from tests.test_verify_step_gpu import _example  # noqa: E402

pytestmark = pytest.mark.gpu


def test_a_tie_with_a_lower_id_is_not_kept():
    """Greedy decoding takes the lowest of the best ids: a drafted one that ties with it is wrong."""
    module, vocab, block = _example(), 1024, 4

    class Tied(module.Verifier):
        def logits(self, tokens, batch):
            x = torch.zeros(tokens.numel(), vocab, dtype=torch.bfloat16, device="cuda")
            x[:, [30, 700]] = 5.0
            return x

    v = Tied(layers=1, hidden=256, Hq=4, Hkv=1, D=64, inner=512, vocab=vocab, seqs=3, max_len=64, page_size=16, group=32)
    draft = torch.tensor([[1, 30, 30, 30], [1, 30, 700, 30], [1, 700, 30, 30]], device="cuda")
    kept, _, top = v.verify(draft.flatten(), None, block)
    assert kept.tolist() == [4, 2, 1]
    assert (top[:, 0] == 30).all() and (top[:, 1] == 700).all()
