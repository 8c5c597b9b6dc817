// tile_out.cuh -- results from TMEM to global rows.
//
// A thread holds a row (TMEM lane) and would store it 16 bytes at a time, a warp touching 32
// rows with every instruction: 3,500 cycles for a 128 x 128 tile.  Instead each warp turns its
// 32 rows through shared memory (rows of 128-byte halves, 16-byte units permuted by the row so
// that no bank is met twice) and stores whole rows, consecutive lanes consecutive bytes.  A
// warp exchanges only its own rows: no barrier but the warp's.
#pragma once
#include "svga_device.cuh"

namespace svga {

// Address of 16-byte unit u of a row in a tile whose 128-byte halves are half_step apart.
__device__ __forceinline__ uint32_t unit_addr(uint32_t tile, uint32_t half_step, int row, int u)
{
    return tile + (u >> 3) * half_step + row * 128 + (((u & 7) ^ (row & 7)) << 4);
}

// NCOL fp32 columns of this lane's TMEM row, times f, as 16-bit values into units u0 and up.
template <int NCOL, bool F16>
__device__ __forceinline__ void put_row_16(uint32_t taddr, uint32_t tile, uint32_t half_step,
                                           int row, int u0, float f, bool any)
{
#pragma unroll 1
    for (int j = 0; j < NCOL / 32; ++j) {
        uint32_t o[32];
        if (any) {
            tmem_ld32(taddr + j * 32, o);
            tmem_wait_ld();
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = pack_16x2<F16>(__uint_as_float(o[8 * c + 2 * i]) * f,
                                      __uint_as_float(o[8 * c + 2 * i + 1]) * f);
            st_shared_v4(unit_addr(tile, half_step, row, u0 + 4 * j + c), x[0], x[1], x[2], x[3]);
        }
    }
}

// NCOL fp32 columns of this lane's TMEM row, times f, in fp32 into units 0 and up.
template <int NCOL>
__device__ __forceinline__ void put_row_32(uint32_t taddr, uint32_t tile, uint32_t half_step,
                                           int row, float f, bool any)
{
#pragma unroll 1
    for (int j = 0; j < NCOL / 32; ++j) {
        uint32_t o[32];
        if (any) {
            tmem_ld32(taddr + j * 32, o);
            tmem_wait_ld();
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            st_shared_v4(unit_addr(tile, half_step, row, 8 * j + c), o[4 * c], o[4 * c + 1],
                         o[4 * c + 2], o[4 * c + 3]);
    }
}

// UNITS 16-byte units from u0 on of the warp's rows row0 .. row0 + valid - 1 to dst (row row0's
// first such byte), `step` bytes from row to row.  Every lane of the warp calls it.
template <int UNITS>
__device__ __forceinline__ void copy_rows_out(uint32_t tile, uint32_t half_step, int row0, int u0,
                                              char *dst, long long step, int valid, int lane)
{
    constexpr int kRows = 32 / UNITS;  // rows an instruction stores
    const int u = lane % UNITS, r = lane / UNITS;
    constexpr int kAtOnce = 32 / kRows < 8 ? 32 / kRows : 8;  // loads before the first store
    __syncwarp();  // the rows are in shared memory
#pragma unroll 1
    for (int i = 0; i < 32; i += kRows * kAtOnce) {
        uint4 x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            ld_shared_v4(unit_addr(tile, half_step, row0 + i + k * kRows + r, u0 + u), x[k].x,
                         x[k].y, x[k].z, x[k].w);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int row = i + k * kRows + r;
            if (row < valid) *reinterpret_cast<uint4 *>(dst + row * step + 16 * u) = x[k];
        }
    }
    __syncwarp();  // and may be overwritten
}

}  // namespace svga
