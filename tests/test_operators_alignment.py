"""Arrays of 4-byte words (tokens, lengths, uniforms, scales, counts, the status word) off their
boundary would fault on the device: the C ABI refuses them with SPEC_EINVAL, without a GPU."""
import pytest

from test_operators_abi import A, LINEAR, P, PROBS, sv  # noqa: F401


@pytest.mark.parametrize("name", ["tokens", "u", "lens", "out", "n", "status"])
@pytest.mark.parametrize("address", [257, 258, 259])
def test_probs(sv, name, address):  # noqa: F811
    assert sv.load_library().spec_verify_probs(*{**PROBS, name: P(address)}.values()) == sv.SPEC_EINVAL


@pytest.mark.parametrize("name", ["xs", "ws", "status"])
@pytest.mark.parametrize("address", [257, 258, 259])
def test_linear(sv, name, address):  # noqa: F811
    args = {**LINEAR, "din": 2, "xs": A, "ws": A, name: P(address)}
    assert sv.load_library().spec_linear(*args.values()) == sv.SPEC_EINVAL
