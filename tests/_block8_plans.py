"""Prefill products of e4m3 codes that a CTA pair works on for several tiles
with several boxes of scales: (M, K, N, tile width, groups of K, rounds of
tiles over 74 pairs).  The width is the library's choice on 148 SMs."""

PIPELINES = [
    (1024, 2176, 8192, 256, 17, 2),
    (1300, 2064, 8208, 256, 17, 3),
    (2048, 4096, 4096, 256, 32, 2),
    (4096, 4112, 2064, 256, 33, 2),
    (4096, 4240, 2064, 256, 34, 2),
    (700, 2176, 8192, 128, 17, 3),
    (2048, 2304, 8192, 128, 18, 7),
    (1025, 4112, 4112, 128, 33, 3),
    (130, 4368, 20480, 128, 35, 3),
    (513, 6160, 20480, 128, 49, 7),
]
