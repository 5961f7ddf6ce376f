"""CPU: limits of the adapter entry points that only very large sizes meet.  Nothing
here is launched."""
import dynamic_mixed_precision_amd as dm
from test_lora_adamw_abi import backward_args, refused


def test_backward_of_a_pool_too_large():
    """More transposed tiles than their launches can count are refused before any launch."""
    big = dict(N=1 << 16, K=1 << 16, n=65535, bytes=1 << 62)
    refused(4, "dmpq_lora_backward", *backward_args(**big))
    assert "2^31" in dm.last_error()
