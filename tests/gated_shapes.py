"""Shapes that reach the kernels of the gated block and of 4-bit weights which smaller ones do not, each
with the kernel that the host rules choose on 256 compute units: test_gated_routes.py asserts that
on the CPU, test_gated_routes_gpu.py runs them."""

F32, F16, BF16 = 0, 1, 2
NAMES = {F32: "f32", F16: "f16", BF16: "bf16"}

# (m, n, k, type): the gated product with 128 x 128 tiles in two stages and in three, whole and ragged
# tiles; the general kernel's large tile in every type, and its small one
FORWARD = {
    (512, 1024, 512, BF16): "LM", (301, 2040, 520, F16): "LM", (700, 520, 200, BF16): "LM",
    (600, 1024, 1600, BF16): "LMD", (577, 1000, 1544, F16): "LMD", (512, 1024, 1536, BF16): "LMD",
    (1100, 1999, 101, F32): "general large", (1100, 1999, 101, BF16): "general large", (1030, 2050, 33, F16): "general large",
    (900, 130, 77, BF16): "general small", (310, 1101, 743, F32): "general small",
}

# (m, d, n, type): the down projection
DOWN = {
    (300, 1000, 520, BF16): "LM", (2040, 2168, 200, F16): "LM", (600, 4096, 1600, BF16): "LMD", (577, 1000, 1544, F16): "LMD",
    (2300, 4104, 264, BF16): "L", (2304, 4096, 256, F16): "L persistent",
    (300, 1100, 743, F32): "general small", (310, 1100, 743, BF16): "general small",
    (2100, 2100, 100, F32): "general large", (2048, 2176, 330, BF16): "general large", (1999, 2222, 99, F16): "general large",
}

# (m, n, k, d, type): kernels of dZ from dY (m, d), of dX, of dW and of the down projection's gradient
BACKWARD = {
    (512, 4096, 64, 2048, BF16): ("LMD", "LMD split", "LM", "LM"),
    (500, 4088, 72, 1608, F16): ("LMD", "LMD split", "LM", "LM"),
    (512, 4096, 64, 512, BF16): ("LM", "LMD split", "LM", "LM"),
    (2048, 2048, 2304, 128, BF16): ("LM", "LW persistent", "L persistent", "LMD"),
    (1100, 4104, 2056, 264, F16): ("LM", "L split", "L", "LM"),
    (2048, 2050, 2100, 2059, F32): ("general large", "general large", "general large", "general large"),
    (2048, 2050, 2051, 2059, BF16): ("general large", "general large", "general large", "general large"),
    (1999, 2222, 2051, 2111, F16): ("general large", "general large", "general large", "general large"),
    (3000, 33, 50, 41, F32): ("general small", "general small", "general small 11 parts", "general small 11 parts"),
    (3000, 33, 50, 41, BF16): ("general small", "general small", "general small 5 parts", "general small 5 parts"),
}

# (m, n, k, group, gated): 4-bit tiles with groups of more than one k-tile of 128: several of a row, the
# last one short, spans of 2, 3, 4, 5
W4 = {
    (700, 1500, 1100, 256, False): "64 x 128", (900, 5000, 1000, 384, False): "128 x 128",
    (900, 2500, 1000, 640, True): "128 x 128", (700, 750, 1152, 512, True): "64 x 128",
    (2100, 8200, 1152, 256, False): "192 x 256", (2100, 8200, 1160, 512, False): "192 x 256",
    (2100, 4100, 1152, 256, True): "192 x 256", (1030, 4104, 1280, 640, True): "192 x 256",
    (2900, 4104, 1000, 384, False): "256 x 256", (2900, 2052, 1000, 384, True): "256 x 256",
    (2900, 4104, 1416, 256, False): "256 x 256",
}
