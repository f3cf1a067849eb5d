"""The attention layer's host-side code (argument checks, workspace layout, the
launches' plans) under AddressSanitizer and UndefinedBehaviorSanitizer, on the
CPU, as the residual block's (test_block_sanitized.py)."""
import test_block_sanitized as block


def test_attention_host_code_under_sanitizers(tmp_path, monkeypatch):
    monkeypatch.setattr(block, "UNDER", ("attn_abi.cpp", "attn_decode.hip"))
    monkeypatch.setattr(block, "TESTS", ("test_attention_abi.py",))
    block.test_block_host_code_under_sanitizers(tmp_path)
