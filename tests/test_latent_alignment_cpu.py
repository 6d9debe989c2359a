"""The C calls of the latent cache refuse arrays of words that do not lie on words: the kernels would fault on them (the
error word of a workspace only when something is flagged).  Nothing is enqueued, so made-up pointers do."""
import pytest

from tests.test_latent_abi_cpu import INVALID, OK_PTR, append, built, sinks, sparse  # noqa: F401


@pytest.mark.parametrize("call,names", [
    (append, ["inv_freq", "table", "off", "vis", "scales", "ws"]),
    (sinks, ["table", "off", "vis", "scales", "lse", "ws"]),
    (sparse, ["table", "off", "vis", "scales", "idx", "lse", "ws"])])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_words_off_their_places_are_refused(call, names, by):
    for name in names:
        assert call(**{name: OK_PTR + by}) == INVALID, name
