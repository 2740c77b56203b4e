"""Shapes of dense_logits_fp8 that between them take every kernel there is, and
the kernel that each takes: (kernel, rows, v, d).  The tiled kernels' workgroups
take tile after tile of several blocks of columns, which these shapes do: more
than 256 tiles, three blocks and more, cut in every direction and not."""

SHAPES = [
    ("tiles 64 128", 31, 66931, 1104),
    ("tiles 64 128", 29, 68655, 512),
    ("tiles 64 128", 409, 9223, 512),
    ("tiles 64 128", 155, 8067, 528),
    ("tiles 64 128", 64, 16000, 2048),
    ("tiles 128 128", 305, 43639, 528),
    ("tiles 128 128", 1442, 10821, 512),
    ("tiles 128 128", 128, 20096, 640),
    ("tiles 64 256", 51, 60013, 1104),
    ("tiles 64 256", 155, 86665, 640),
    ("tiles 64 256", 319, 45301, 400),
    ("tiles 64 256", 40, 65536, 1152),
    ("tiles 128 256", 1525, 13383, 1104),
    ("tiles 128 256", 579, 16647, 512),
    ("tiles 128 256", 146, 48333, 400),
    ("tiles 128 256", 512, 32768, 640),
    ("rows 32 64", 387, 4863, 400),
    ("rows 32 64", 796, 2477, 512),
    ("rows 32 64", 17, 5003, 1104),
    ("rows 16 64", 9, 20003, 400),
    ("rows 16 64", 16, 40001, 512),
    ("rows 16 32", 1, 20003, 400),
    ("rows 16 32", 4, 40003, 640),
    ("rows 16 32", 16, 9001, 1104),
    ("rows 16 16", 1, 5003, 400),
    ("rows 16 16", 15, 4001, 512),
]

# rows of out too far apart for the tiles' offsets: elements of fp32, of bf16
FAR = ("rows 32 64", 70, 20000, 512, {4: 1 << 21, 2: 1 << 22})


def ldo(v: int, size: int) -> int:
    """The smallest stride of rows of v values that start at multiples of 16 bytes."""
    return -(-v * size // 16) * 16 // size
