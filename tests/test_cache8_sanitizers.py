"""The host code of the rotary positions and the 8-bit cache under AddressSanitizer and UndefinedBehaviorSanitizer (CPU):
as test_hybrid_sanitizers, with the files and tests of these operators."""
import test_hybrid_sanitizers as base


def test_cache8_host_code_under_asan_ubsan(tmp_path, monkeypatch):
    monkeypatch.setattr(base, "CHECKED", ["api.cpp", "api_hybrid.cpp", "rotary.hip", "cache8.hip", "attn_cached8.hip", "check.hip"])
    monkeypatch.setattr(base, "TESTS", ["tests/test_cache8_abi.py", "tests/test_cache8_binding.py"])
    base.test_hybrid_host_code_under_asan_ubsan(tmp_path)
