"""The host-side argument checks of the gated delta rule, the convolution on a cache
and the layer norm under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only, no
GPU call), as test_block_abi_sanitized.py runs those of the SSD layer's operators."""
import test_block_abi_sanitized as block


def test_delta_host_checks_under_asan_and_ubsan(tmp_path, monkeypatch):
    monkeypatch.setattr(block, "FILES", ("test_delta_abi_host.py",))
    block.test_block_host_checks_under_asan_and_ubsan(tmp_path)
