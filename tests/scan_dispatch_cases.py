"""Prompt batches with the launches that the scan takes them in: tests/test_scan_dispatch.py
holds the calls' plan to this, tests/test_gpu_scan_dispatch.py their results.
A case: heads, groups, dk, dv, type, lengths, launches.  Launches: "step" (token by token, up to the
length behind it), "chunks" (those longer than the length behind it), each with the
tokens of a segment (0: whole) and, in segments, who joins them."""

DRAFTS = [5] * 64
CASES = {
    # both launches, prompts on both sides of 24 tokens
    "both": (4, 2, 128, 64, "bf16", [24, 25, 1, 0, 130, 5, 3, 2, 7, 23, 26, 4], ["chunks 24 0", "step 24 0"]),
    "both_128": (5, 1, 128, 128, "bf16", [24, 25, 1, 0, 130, 5, 3, 2, 7, 23, 26, 4], ["chunks 24 0", "step 24 0"]),
    "both_64": (11, 1, 64, 64, "bf16", [0, 0, 64, 1, 24, 25, 2, 3, 0, 65, 1, 1, 2], ["chunks 24 0", "step 24 0"]),
    # .. and more prompts than a wave has lanes
    "both_many": (4, 2, 128, 64, "bf16", DRAFTS[:30] + [25, 300, 0, 64] + DRAFTS[30:] + [65, 24, 26, 129, 100, 1], ["chunks 24 0", "step 24 0"]),
    "drafts": (4, 2, 64, 64, "bf16", DRAFTS + [5] * 9, ["chunks 24 0", "step 24 0"]),
    # one launch of chunks, more than 64 prompts
    "chunks_many": (3, 1, 64, 64, "bf16", [(37 * i) % 131 for i in range(75)], ["chunks -1 0"]),
    # segments of 128 tokens of more than 64 prompts
    "segments_many": (4, 1, 64, 64, "bf16", [4] * 40 + [9000] + [0, 3] * 12 + [8800], ["chunks -1 128 launch"]),
    # segments of 256 tokens and more: chained, and joined by a launch
    "segments_256": (32, 32, 64, 64, "bf16", [1100], ["chunks -1 256 each"]),
    "segments_256_wide": (24, 24, 128, 128, "bf16", [1400], ["chunks -1 256 each"]),
    "segments_256_joined": (16, 16, 64, 64, "bf16", [3000, 1333], ["chunks -1 256 launch"]),
    "segments_512": (16, 16, 64, 64, "bf16", [4999], ["chunks -1 512 launch"]),
    "segments_512_wide": (16, 16, 128, 64, "bf16", [4421], ["chunks -1 512 launch"]),
    # token by token in segments, more than 64 prompts
    "step_segments_many": (2, 1, 64, 64, "f32", [3] * 50 + [6000, 0] + [2] * 17 + [6200], ["step all 32 launch"]),
    "step_segments_16": (3, 3, 16, 32, "bf16", [2500, 700], ["step all 32 launch"]),
    "step_whole": (40, 8, 128, 64, "f32", [70, 130, 24, 25, 1], ["step all 0"]),
}
