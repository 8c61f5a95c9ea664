"""GPU: calls at the limits of what the operators around a prefix cache allow."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_ops import BF, F32, TYPES, Rand  # noqa: F401
from test_gpu_prefix import draw_check, settings

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import gated_deltanet_state_gdn_amd as gdn
    gdn.load()
    yield


def G():
    import gated_deltanet_state_gdn_amd as gdn
    return gdn


# ------------------------------------------------------------------ the next token
@TYPES
@pytest.mark.parametrize("width", [32768, 131072])
def test_sample_flat_rows_with_loose_ends(dt, width):
    # every token of the row is about the border, whole 16-byte pieces reach to its end, and elements lie in front of the
    # first one: the last turn of looking the row through lists 16 tokens a thread and the ends
    us = [0.0, 0.25, 0.51, 0.9, 1.0 - 2.0 ** -24]
    u = torch.tensor(us, device="cuda")
    for offset in (1, 2, 3):
        x = torch.zeros(5, width, dtype=dt, device="cuda")[:, offset:]
        vocab = width - offset
        say("flat", dt, width, offset)
        # equal weights: token j is the first with j + 1 > u n, n tokens staying
        for kw, n in ((dict(), vocab), (dict(k=vocab - 5), vocab - 5), (dict(k=vocab // 2), vocab // 2), (dict(T=100.0, p=0.5), -(-vocab // 2)), (dict(m=0.5), vocab)):
            token = G().gdn_sample(x, u, **settings(5, **kw))
            want = [int(v * n) for v in u.double().tolist()]
            assert token.tolist() == want, (dt, width, offset, kw)
    # a temperature at which all tokens are of one bin
    x = Rand(width).n(5, width, scale=2.0).to(dt)[:, 1:]
    for kw in (dict(), dict(k=width // 2, p=0.7)):
        draw_check(x, u, settings(5, T=1e30, **kw), 0.0)


@TYPES
def test_sample_flat_rows_of_odd_length(dt):
    # contiguous rows, of which each starts at another place in 16 bytes
    u = torch.linspace(0.0, 0.99, 9).cuda()
    for vocab in (32767, 32761, 49151):
        x = torch.zeros(9, vocab, dtype=dt, device="cuda")
        say("flat", dt, vocab)
        assert G().gdn_sample(x, u).tolist() == [int(v * vocab) for v in u.double().tolist()]
