"""Host-side rules of the key/value cache's binding that need no GPU."""
import pytest

from sparse_depth_token_gb300 import xmod as X

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("which", ["q_norm", "k_norm"])
def test_gains_have_to_be_contiguous(which):
    hd = 64
    both = torch.ones(hd, 2, dtype=torch.bfloat16)
    # one element, expanded, counts hd elements but stores one
    bad = [both[:, 0], both[:1, 0].expand(hd), both[:, 0].contiguous().float(), both[:hd - 1, 0].contiguous()]
    for gain in bad:
        with pytest.raises(X.XmodError) as e:
            X._check_gains("xmod_cache_append", X.layer_weights({which: gain}), torch.bfloat16, hd, -1)
        assert e.value.status == X.ERR_INVALID_ARG
    good = both[:, 0].contiguous()
    X._check_gains("xmod_cache_append", X.layer_weights({which: good}), torch.bfloat16, hd, -1)
    X._check_gains("xmod_cache_append", X.layer_weights({which: good.view(1, hd)}), torch.bfloat16, hd, -1)
    X._check_gains("xmod_cache_append", X.layer_weights({}), torch.bfloat16, hd, -1)
    X._check_gains("xmod_cache_append", None, torch.bfloat16, hd, -1)
