// pages_params.cuh -- parameters of the page kernels (pages.cu).
#pragma once
#include <stdint.h>

#include "kda_device.cuh"
#include "launch_order.cuh"

namespace kda {

constexpr int PG_MAX_ROWS = 65536;  // rows of a table: a bit each in shared memory
constexpr int PG_MAX_COPY = 1 << 21;  // pairs of one copy: every block looks through them all, once for each 1024 of its own
constexpr int PG_MAX_LIST = 8192;   // sequences of one reserve or fork: their prefix sums lie in shared memory

struct PagesParams {
    int *table, *length, *ref;       // [R][P], [R], [num_pages]
    const int *rows, *src, *new_length;  // [n]; src: fork, new_length: reserve
    int *copy_src, *copy_dst;        // [n]: fork's copies
    int *table_out, *ref_out;        // compact
    int *info;                       // [1] or NULL
    int *ws_counts, *ws_n, *ws_hole, *ws_move, *ws_rank;  // compact's workspace
    int n, R, P, num_pages, ps;
    DeviceStatus st;
};

struct PoolParams {
    uint8_t *pool;
    const int *src, *dst, *count;    // count: pairs, on the device, or NULL
    long long outer, outer_stride, page_stride, page_bytes;
    int num_pages, n, unit;          // unit: bytes that a block copies at a time
    DeviceStatus st;
};

}  // namespace kda
