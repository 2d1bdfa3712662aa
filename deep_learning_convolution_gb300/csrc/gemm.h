// gemm.h -- what gemm.cu and gemm_rows.cu share on the host.
#pragma once

#include "internal.h"

struct FewRowsPlan {
    int num_kb, rows, filters, filter_tiles, row_tiles, splits;  // filters: outputs of a tile
    double us;  // expected time
};

// gemm_rows.cu: operands as TMA loads them (see gemm.cu's packing).
FewRowsPlan dlc_few_rows_plan(const dlcContext *ctx, const GemmProblem &g);
dlcStatus_t dlc_launch_few_rows(dlcContext *ctx, const GemmProblem &g);

// gemv.cu: a few rows on the CUDA cores, operands as they are.  Whether it is
// the faster way, and the launch.
bool dlc_gemv_ok(const GemmProblem &g);
dlcStatus_t dlc_launch_gemv(dlcContext *ctx, const GemmProblem &g);

// gemm.cu: a row operand's tensor map.
bool dlc_encode_operand(const dlcContext *ctx, CUtensorMap *tm, const GemmOperand &o, long long rows, int ch, int box_rows);

// Whether every row starts on a boundary of four elements, channels contiguous.
inline bool dlc_vec4_rows(const RowTensor &t) {
    if (!t.p) return true;
    const long long e = dlc_dtype_bytes((dlcDataType_t)t.dt);
    auto mult = [&](long long s) { return (s * e) % (4 * e) == 0; };
    return t.m.cs == 1 && (uintptr_t)t.p % (4 * e) == 0 &&
           (t.m.uniform ? mult(t.m.ld) : (mult(t.m.s0) && mult(t.m.s2) && mult(t.m.s3)));
}
