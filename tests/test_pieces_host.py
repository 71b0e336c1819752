"""Launches of many blocks go out in pieces that the grid's limits allow."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_pieces_cover_every_block(tmp_path):
    exe = str(tmp_path / "pieces_driver")
    subprocess.run(["g++", "-O2", "-std=c++17", os.path.join(HERE, "pieces_driver.cpp"), "-o", exe], check=True)
    # 65536 groups of 4096 rows, four to a block; a 65536 x 65536 matrix, 256 entries to a block
    sizes = [0, 1, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 65536 * 4096 // 4, 65536 * 65536 // 256, 2 ** 31 + 7, 2 ** 36]
    out = subprocess.run([exe, *map(str, sizes)], capture_output=True, text=True, check=True).stdout.split("\n")
    for size, line in zip(sizes, out):
        pieces, whole, most = map(int, line.split())
        assert whole == 1 and most * 512 < 2 ** 32 and pieces == -(-size // 2 ** 22)
