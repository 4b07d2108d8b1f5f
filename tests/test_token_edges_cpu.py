"""Refusals of the token-step operators beside those of test_token_ops_cpu.py."""
from test_token_ops_cpu import BAD, L, norm, refused  # noqa: F401


def test_norm_refuses_one_memory_for_both_outputs(L):  # noqa: F811
    refused(L, BAD, norm(L, y=32, total=32, ldt=64), "same memory")
    refused(L, BAD, norm(L, y=32, total=48, ldt=64), "handle is NULL")
    refused(L, BAD, norm(L, x=32, y=32), "handle is NULL")
    refused(L, BAD, norm(L, x=32, y=48, total=32, ldt=64), "handle is NULL")
