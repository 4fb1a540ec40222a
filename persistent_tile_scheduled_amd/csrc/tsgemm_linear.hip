// C ABI of the gated projection and of the linear head's cross entropy
// (include/tsgemm.h): argument checks and launches.  Conventions as in tsgemm.hip.
#include <hip/hip_runtime.h>

#include "tsgemm_checks.h"
#include "tsgemm_linear_kernel.h"
#include "tsgemm_linear_launch.h"
#include "tsgemm_linear_rows.h"
#include "tsgemm_linear_shape.h"

namespace {

using namespace tsg;

constexpr int64_t kMostStride = int64_t(1) << 23;  // 32-bit offsets in a quarter of a slab
constexpr uint32_t kNoHalf = 0xFFFFFFFFu;

int check_16bit(int dt) {
    if (dt != TSGEMM_FP16 && dt != TSGEMM_BF16) return fail(TSGEMM_EINVAL, "dtype must be TSGEMM_FP16 (1) or TSGEMM_BF16 (2), got %d", dt);
    return TSGEMM_OK;
}
int check_act(int act) {
    if (act < TSGEMM_SILU || act > TSGEMM_GELU_TANH)
        return fail(TSGEMM_EINVAL, "act must be TSGEMM_SILU (1), TSGEMM_GELU (2) or TSGEMM_GELU_TANH (3), got %d", act);
    return TSGEMM_OK;
}
// rows, width and the other side's size (of hidden or vocab)
int check_linear(int64_t rows, int64_t other, const char* what, int64_t width) {
    const int rc = check_shape(rows, width);
    if (rc != TSGEMM_OK) return rc;
    if (width < 8 || width % 8 != 0) return fail(TSGEMM_EINVAL, "width must be a positive multiple of 8 (16-byte rows), got %lld", (long long)width);
    if (other < 0 || other >= (int64_t(1) << 31)) return fail(TSGEMM_EINVAL, "%s must be in [0, 2^31)", what);
    if (width >= kMostStride || other >= (int64_t(1) << 30))
        return fail(TSGEMM_EUNSUPPORTED, "width must be below 2^23 and %s below 2^30", what);
    return TSGEMM_OK;
}
// A product's operand: rows of 16-byte aligned chunks.
int check_operand(const char* name, const void* p, int64_t ld, int64_t width) {
    const int rc = check_matrix(name, p, ld, width, TSGEMM_BF16);
    if (rc != TSGEMM_OK) return rc;
    if (off(p, 16) || ld % 8 != 0) return fail(TSGEMM_EINVAL, "the rows of %s must be 16-byte aligned", name);
    if (ld >= kMostStride) return fail(TSGEMM_EUNSUPPORTED, "the row stride of %s must be below 2^23", name);
    return TSGEMM_OK;
}
int check_tiles(const LinShape& s) {
    if (s.m_blocks * s.n_blocks * s.splits >= (int64_t(1) << 31)) return fail(TSGEMM_EUNSUPPORTED, "too many tiles");
    return TSGEMM_OK;
}

template <class F>
void of_type(int dt, F&& f) {
    if (dt == TSGEMM_FP16) f(LinearOf<TSGEMM_FP16>{});
    else f(LinearOf<TSGEMM_BF16>{});
}

LinArgs product(const LinShape& s, int64_t M, int64_t N) {
    LinArgs a = {};
    a.M = (uint32_t)M; a.N = (uint32_t)N;
    a.m_blocks = (uint32_t)s.m_blocks; a.n_blocks = (uint32_t)s.n_blocks;
    a.splits = (uint32_t)s.splits; a.slabs = (uint32_t)s.slabs; a.slabs_per_split = (uint32_t)s.per_split;
    a.seg_slabs = a.half = kNoHalf;
    return a;
}
LinSumArgs sum_of(const LinArgs& a, const float* sums) {
    LinSumArgs s = {};
    s.sums = sums; s.splits = a.splits; s.M = a.M; s.N = a.N; s.out = a.out; s.out2 = a.out2;
    s.ldo = a.ldo; s.ldo2 = a.ldo2; s.half = a.half; s.out_rows = a.out_rows; s.unscale = a.unscale;
    return s;
}
int64_t slabs_of(int64_t n) { return (n + 63) / 64; }
int64_t aligned(int64_t bytes) { return round_up(bytes, 256); }

// The gated gradient's products and where they lie in the workspace.
struct GatedGradPlan {
    LinShape dx, dw;
    int64_t pitch, ld, sums, bytes;  // sums: of either product, one after the other
    GatedGradPlan(int64_t rows, int64_t hidden, int64_t width) {
        pitch = gated_pitch(hidden);
        dx = linear_shape(rows, width, 2 * slabs_of(hidden), false, true);
        dw = linear_shape(2 * pitch, width, slabs_of(rows), false, true);
        const int64_t x = dx.splits > 1 ? dx.splits * rows * width * 4 : 0, w = dw.splits > 1 ? dw.splits * 2 * pitch * width * 4 : 0;
        ld = 2 * pitch;
        sums = aligned(rows * ld * 2);
        bytes = sums + aligned(x > w ? x : w);
    }
};

struct LossPlan {
    LinShape s;
    bool few;
    int64_t parts, hit, bytes;
    LossPlan(int64_t rows, int64_t vocab, int64_t width) {
        s = linear_shape(rows, vocab, slabs_of(width), false, false);
        few = takes_few(s, rows, vocab, width, 1);
        parts = few ? few_groups(vocab) : 2 * s.n_blocks;
        hit = aligned(parts * rows * 8);
        bytes = hit + aligned(rows * 4);
    }
};

struct LossGradPlan {
    int64_t piece, ld, ldx, unscale, x, dl, dx_sums, dw_sums, bytes;
    LinShape logits, dx, dw;  // of a whole piece
    LossGradPlan(int64_t rows, int64_t vocab, int64_t width) {
        piece = vocab_piece(rows, vocab);
        logits = linear_shape(rows, piece, slabs_of(width), false, false);
        dx = linear_shape(rows, width, piece / 64, false, true);
        dw = linear_shape(piece, width, slabs_of(rows), false, true);
        unscale = aligned(rows * 16);
        ld = piece;
        ldx = width;
        x = unscale + 256;
        dl = x + aligned(rows * ldx * 2);
        dx_sums = dl + aligned(rows * ld * 2);
        dw_sums = dx_sums + (dx.splits > 1 || vocab > piece ? aligned(dx.splits * rows * width * 4) : 0);
        bytes = dw_sums + (dw.splits > 1 ? aligned(dw.splits * piece * width * 4) : 0);
    }
};

// every call's sizes fit 63 bits and every product's tiles 31
int check_volume(int64_t rows, int64_t other, int64_t width) {
    if ((__int128)rows * other >= (__int128(1) << 40) || (__int128)rows * width >= (__int128(1) << 40) ||
        (__int128)other * width >= (__int128(1) << 40))
        return fail(TSGEMM_EUNSUPPORTED, "a matrix of 2^40 values or more");
    return TSGEMM_OK;
}

}  // namespace

extern "C" {

int tsgemm_gated_linear(int64_t rows, int64_t hidden, int64_t width, int dtype, int act, const void* x, int64_t ldx,
                        const void* gate_weight, int64_t ldgw, const void* up_weight, int64_t lduw, void* y, int64_t ldy,
                        void* gate, int64_t ldgate, void* up, int64_t ldup, void* stream) {
    reset_error();
    int rc = check_linear(rows, hidden, "hidden", width);
    if (rc == TSGEMM_OK) rc = check_volume(rows, hidden, width);
    if (rc == TSGEMM_OK) rc = check_16bit(dtype);
    if (rc == TSGEMM_OK) rc = check_act(act);
    if (rc != TSGEMM_OK || rows == 0 || hidden == 0) return rc;
    rc = check_operand("x", x, ldx, width);
    if (rc == TSGEMM_OK) rc = check_operand("gate_weight", gate_weight, ldgw, width);
    if (rc == TSGEMM_OK) rc = check_operand("up_weight", up_weight, lduw, width);
    if (rc == TSGEMM_OK) rc = check_matrix("y", y, ldy, hidden, dtype);
    if (rc == TSGEMM_OK && gate) rc = check_matrix("gate", gate, ldgate, hidden, dtype);
    if (rc == TSGEMM_OK && up) rc = check_matrix("up", up, ldup, hidden, dtype);
    if (rc == TSGEMM_OK)
        rc = check_overlaps({matrix("y", y, rows, hidden, ldy, 2), matrix("gate", gate, rows, hidden, ldgate, 2),
                             matrix("up", up, rows, hidden, ldup, 2)},
                            {matrix("x", x, rows, width, ldx, 2), matrix("gate_weight", gate_weight, hidden, width, ldgw, 2),
                             matrix("up_weight", up_weight, hidden, width, lduw, 2)});
    if (rc != TSGEMM_OK) return rc;
    const LinShape s = linear_shape(rows, hidden, slabs_of(width), true, false);
    rc = check_tiles(s);
    if (rc != TSGEMM_OK) return rc;
    LinArgs a = product(s, rows, hidden);
    a.a = static_cast<const uint16_t*>(x); a.lda = ldx;
    a.b = static_cast<const uint16_t*>(gate_weight); a.ldb = ldgw;
    a.b2 = static_cast<const uint16_t*>(up_weight); a.ldb2 = lduw;
    a.Ka = a.Kb = (uint32_t)width;
    a.y = static_cast<uint16_t*>(y); a.gate = static_cast<uint16_t*>(gate); a.up = static_cast<uint16_t*>(up);
    a.ldy = ldy; a.ldgate = ldgate; a.ldup = ldup; a.act = act;
    a.aligned = !off(y, 16) && ldy % 8 == 0 && (!gate || (!off(gate, 16) && ldgate % 8 == 0)) && (!up || (!off(up, 16) && ldup % 8 == 0));
    (void)hipGetLastError();
    of_type(dtype, [&](auto k) {
        if (takes_few(s, rows, hidden, width, 2)) k.few(LIN_KIND_GATED, a, static_cast<hipStream_t>(stream));
        else k.product(LIN_KIND_GATED, s.tile, a, static_cast<hipStream_t>(stream));
    });
    return launched("gated linear");
}

int64_t tsgemm_gated_linear_grad_workspace(int64_t rows, int64_t hidden, int64_t width) {
    reset_error();
    int rc = check_linear(rows, hidden, "hidden", width);
    if (rc == TSGEMM_OK) rc = check_volume(rows, hidden, width);
    if (rc == TSGEMM_OK && 2 * gated_pitch(hidden) >= kMostStride) rc = fail(TSGEMM_EUNSUPPORTED, "hidden must be below 2^22");
    if (rc != TSGEMM_OK) return rc;
    return rows == 0 || hidden == 0 ? 0 : GatedGradPlan(rows, hidden, width).bytes;
}

int tsgemm_gated_linear_grad(int64_t rows, int64_t hidden, int64_t width, int dtype, int act, const void* dy, int64_t lddy,
                             const void* x, int64_t ldx, const void* gate_weight, int64_t ldgw, const void* up_weight,
                             int64_t lduw, const void* gate, int64_t ldgate, const void* up, int64_t ldup, void* dx,
                             int64_t lddx, void* dgate_weight, int64_t lddgw, void* dup_weight, int64_t ldduw, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    const int64_t need = tsgemm_gated_linear_grad_workspace(rows, hidden, width);
    if (need < 0) return (int)need;
    int rc = check_16bit(dtype);
    if (rc == TSGEMM_OK) rc = check_act(act);
    if (rc != TSGEMM_OK) return rc;
    if (!dgate_weight != !dup_weight) return fail(TSGEMM_EINVAL, "dgate_weight and dup_weight are given together or not at all");
    if (!dx && !dgate_weight) return fail(TSGEMM_EINVAL, "no output: dx, or dgate_weight and dup_weight, must be given");
    if (dx && rows > 0) rc = check_operand("dx", dx, lddx, width);
    if (rc == TSGEMM_OK && dgate_weight && hidden > 0) {
        rc = check_operand("dgate_weight", dgate_weight, lddgw, width);
        if (rc == TSGEMM_OK) rc = check_operand("dup_weight", dup_weight, ldduw, width);
    }
    if (rc != TSGEMM_OK) return rc;
    const bool some = rows > 0 && hidden > 0;
    if (some) {
        rc = check_matrix("dy", dy, lddy, hidden, dtype);
        if (rc == TSGEMM_OK) rc = check_operand("x", x, ldx, width);
        if (rc == TSGEMM_OK) rc = check_operand("gate_weight", gate_weight, ldgw, width);
        if (rc == TSGEMM_OK) rc = check_operand("up_weight", up_weight, lduw, width);
        if (rc == TSGEMM_OK) rc = check_matrix("gate", gate, ldgate, hidden, dtype);
        if (rc == TSGEMM_OK) rc = check_matrix("up", up, ldup, hidden, dtype);
        if (rc != TSGEMM_OK) return rc;
        if (!workspace || off(workspace, 16) || workspace_bytes < need)
            return fail(TSGEMM_EINVAL, "this shape needs a 16-byte aligned workspace of %lld bytes", (long long)need);
    }
    rc = check_overlaps({matrix("dx", dx, rows, width, lddx, 2), matrix("dgate_weight", dgate_weight, hidden, width, lddgw, 2),
                         matrix("dup_weight", dup_weight, hidden, width, ldduw, 2), stretch("workspace", workspace, need)},
                        {matrix("dy", some ? dy : nullptr, rows, hidden, lddy, 2), matrix("x", some ? x : nullptr, rows, width, ldx, 2),
                         matrix("gate_weight", some ? gate_weight : nullptr, hidden, width, ldgw, 2),
                         matrix("up_weight", some ? up_weight : nullptr, hidden, width, lduw, 2),
                         matrix("gate", some ? gate : nullptr, rows, hidden, ldgate, 2),
                         matrix("up", some ? up : nullptr, rows, hidden, ldup, 2)});
    if (rc != TSGEMM_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint16_t* const out_dx = static_cast<uint16_t*>(dx);
    uint16_t* const out_dg = static_cast<uint16_t*>(dgate_weight);
    uint16_t* const out_du = static_cast<uint16_t*>(dup_weight);
    if (!some && !(dx && rows > 0) && !(dgate_weight && hidden > 0)) return TSGEMM_OK;
    (void)hipGetLastError();
    if (!some) {  // empty sums
        if (dx && rows > 0) launch_linear_zero(out_dx, lddx, rows, (uint32_t)width, s);
        if (out_dg && hidden > 0) {
            launch_linear_zero(out_dg, lddgw, hidden, (uint32_t)width, s);
            launch_linear_zero(out_du, ldduw, hidden, (uint32_t)width, s);
        }
        return launched("gated linear gradient");
    }
    const GatedGradPlan plan(rows, hidden, width);
    rc = check_tiles(plan.dx);
    if (rc == TSGEMM_OK) rc = check_tiles(plan.dw);
    if (rc != TSGEMM_OK) return rc;
    uint16_t* const d = static_cast<uint16_t*>(workspace);
    float* const sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.sums);

    GatedGradArgs g = {};
    g.dy = static_cast<const uint16_t*>(dy); g.gate = static_cast<const uint16_t*>(gate); g.up = static_cast<const uint16_t*>(up);
    g.d = d; g.lddy = lddy; g.ldgate = ldgate; g.ldup = ldup; g.rows = rows; g.act = act;
    g.hidden = (uint32_t)hidden; g.filled = (uint32_t)round_up(hidden, 64); g.pitch = (uint32_t)plan.pitch; g.ld = plan.ld;
    of_type(dtype, [&](auto k) { k.gated_slope(g, s); });
    rc = launched("gated linear gradient");
    if (rc != TSGEMM_OK) return rc;
    if (dx) {
        LinArgs a = product(plan.dx, rows, width);
        a.a = d; a.a2 = d + plan.pitch; a.lda = plan.ld; a.Ka = g.filled;
        a.b = static_cast<const uint16_t*>(gate_weight); a.ldb = ldgw;
        a.b2 = static_cast<const uint16_t*>(up_weight); a.ldb2 = lduw; a.Kb = (uint32_t)hidden;
        a.seg_slabs = (uint32_t)slabs_of(hidden);
        a.out = out_dx; a.ldo = lddx; a.out_rows = (uint32_t)rows;
        a.sums = plan.dx.splits > 1 ? sums : nullptr;
        of_type(dtype, [&](auto k) {
            k.product(LIN_KIND_DX, plan.dx.tile, a, s);
            if (a.sums) k.sum(sum_of(a, sums), s);
        });
        rc = launched("gated linear gradient of x");
        if (rc != TSGEMM_OK) return rc;
    }
    if (out_dg) {
        LinArgs a = product(plan.dw, 2 * plan.pitch, width);
        a.a = d; a.lda = plan.ld; a.Ka = a.Kb = (uint32_t)rows;
        a.b = static_cast<const uint16_t*>(x); a.ldb = ldx;
        a.out = out_dg; a.ldo = lddgw; a.out2 = out_du; a.ldo2 = ldduw;
        a.half = (uint32_t)plan.pitch; a.out_rows = (uint32_t)hidden;
        a.sums = plan.dw.splits > 1 ? sums : nullptr;
        of_type(dtype, [&](auto k) {
            k.product(LIN_KIND_DW, plan.dw.tile, a, s);
            if (a.sums) k.sum(sum_of(a, sums), s);
        });
        rc = launched("gated linear gradient of the weights");
    }
    return rc;
}

int64_t tsgemm_linear_cross_entropy_workspace(int64_t rows, int64_t vocab, int64_t width) {
    reset_error();
    int rc = check_linear(rows, vocab, "vocab", width);
    if (rc == TSGEMM_OK) rc = check_volume(rows, vocab, width);
    if (rc == TSGEMM_OK && vocab < 1) rc = fail(TSGEMM_EINVAL, "the cross entropy needs a vocabulary of at least 1");
    if (rc != TSGEMM_OK) return rc;
    return rows == 0 ? 0 : LossPlan(rows, vocab, width).bytes;
}

int tsgemm_linear_cross_entropy(int64_t rows, int64_t vocab, int64_t width, int dtype, const void* x, int64_t ldx,
                                const void* weight, int64_t ldw, const int64_t* target, int64_t ignore_index, float* loss,
                                float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = tsgemm_linear_cross_entropy_workspace(rows, vocab, width);
    if (need < 0) return (int)need;
    int rc = check_16bit(dtype);
    if (rc != TSGEMM_OK || rows == 0) return rc;
    rc = check_operand("x", x, ldx, width);
    if (rc == TSGEMM_OK) rc = check_operand("weight", weight, ldw, width);
    if (rc != TSGEMM_OK) return rc;
    if (!target || !loss || !lse || off(target, 8) || off(loss, 4) || off(lse, 4))
        return fail(TSGEMM_EINVAL, "target, loss and lse must be given, aligned to their types");
    if (!workspace || off(workspace, 16) || workspace_bytes < need)
        return fail(TSGEMM_EINVAL, "this shape needs a 16-byte aligned workspace of %lld bytes", (long long)need);
    rc = check_overlaps({stretch("loss", loss, 4 * rows), stretch("lse", lse, 4 * rows), stretch("workspace", workspace, need)},
                        {matrix("x", x, rows, width, ldx, 2), matrix("weight", weight, vocab, width, ldw, 2),
                         stretch("target", target, 8 * rows)});
    if (rc != TSGEMM_OK) return rc;
    const LossPlan plan(rows, vocab, width);
    rc = check_tiles(plan.s);
    if (rc != TSGEMM_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    LinArgs a = product(plan.s, rows, vocab);
    a.a = static_cast<const uint16_t*>(x); a.lda = ldx;
    a.b = static_cast<const uint16_t*>(weight); a.ldb = ldw;
    a.Ka = a.Kb = (uint32_t)width;
    a.target = target;
    a.part = static_cast<float2*>(workspace);
    a.hit = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.hit);
    (void)hipGetLastError();
    of_type(dtype, [&](auto k) {
        if (plan.few) k.few(LIN_KIND_LSE, a, s);
        else k.product(LIN_KIND_LSE, plan.s.tile, a, s);
    });
    rc = launched("linear cross entropy");
    if (rc != TSGEMM_OK) return rc;
    LossArgs j = {};
    j.part = a.part; j.hit = a.hit; j.target = target; j.loss = loss; j.lse = lse; j.ignore = ignore_index;
    j.rows = rows; j.parts = (uint32_t)plan.parts; j.vocab = (uint32_t)vocab;
    launch_loss_join(j, s);
    return launched("linear cross entropy join");
}

int64_t tsgemm_linear_cross_entropy_grad_workspace(int64_t rows, int64_t vocab, int64_t width) {
    reset_error();
    int rc = check_linear(rows, vocab, "vocab", width);
    if (rc == TSGEMM_OK) rc = check_volume(rows, vocab, width);
    if (rc == TSGEMM_OK && vocab < 1) rc = fail(TSGEMM_EINVAL, "the cross entropy needs a vocabulary of at least 1");
    if (rc != TSGEMM_OK) return rc;
    return rows == 0 ? 0 : LossGradPlan(rows, vocab, width).bytes;
}

int tsgemm_linear_cross_entropy_grad(int64_t rows, int64_t vocab, int64_t width, int dtype, const float* dloss, const void* x,
                                     int64_t ldx, const void* weight, int64_t ldw, const int64_t* target,
                                     int64_t ignore_index, const float* lse, void* dx, int64_t lddx, void* dweight,
                                     int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = tsgemm_linear_cross_entropy_grad_workspace(rows, vocab, width);
    if (need < 0) return (int)need;
    int rc = check_16bit(dtype);
    if (rc != TSGEMM_OK) return rc;
    if (!dx && !dweight) return fail(TSGEMM_EINVAL, "no output: dx or dweight must be given");
    if (dx && rows > 0) rc = check_operand("dx", dx, lddx, width);
    if (rc == TSGEMM_OK && dweight) rc = check_operand("dweight", dweight, lddw, width);
    if (rc != TSGEMM_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint16_t* const out_dx = static_cast<uint16_t*>(dx);
    uint16_t* const out_dw = static_cast<uint16_t*>(dweight);
    if (rows == 0) {
        if (!dweight) return TSGEMM_OK;
        (void)hipGetLastError();
        launch_linear_zero(out_dw, lddw, vocab, (uint32_t)width, s);
        return launched("linear cross entropy gradient");
    }
    rc = check_operand("x", x, ldx, width);
    if (rc == TSGEMM_OK) rc = check_operand("weight", weight, ldw, width);
    if (rc != TSGEMM_OK) return rc;
    if (!target || !dloss || !lse || off(target, 8) || off(dloss, 4) || off(lse, 4))
        return fail(TSGEMM_EINVAL, "target, dloss and lse must be given, aligned to their types");
    if (!workspace || off(workspace, 16) || workspace_bytes < need)
        return fail(TSGEMM_EINVAL, "this shape needs a 16-byte aligned workspace of %lld bytes", (long long)need);
    rc = check_overlaps({matrix("dx", dx, rows, width, lddx, 2), matrix("dweight", dweight, vocab, width, lddw, 2),
                         stretch("workspace", workspace, need)},
                        {matrix("x", x, rows, width, ldx, 2), matrix("weight", weight, vocab, width, ldw, 2),
                         stretch("target", target, 8 * rows), stretch("dloss", dloss, 4 * rows), stretch("lse", lse, 4 * rows)});
    if (rc != TSGEMM_OK) return rc;
    const LossGradPlan plan(rows, vocab, width);
    for (const LinShape* p : {&plan.logits, &plan.dx, &plan.dw})
        if ((rc = check_tiles(*p)) != TSGEMM_OK) return rc;
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    uint16_t* const dl = reinterpret_cast<uint16_t*>(w + plan.dl);

    LossGradArgs g = {};
    g.dloss = dloss; g.lse = lse; g.target = target; g.x = static_cast<const uint16_t*>(x); g.ldx = ldx;
    g.counted_x = dweight ? reinterpret_cast<uint16_t*>(w + plan.x) : nullptr;
    g.row = reinterpret_cast<LossRow*>(w); g.unscale = reinterpret_cast<float*>(w + plan.unscale);
    g.ldcx = plan.ldx; g.ignore = ignore_index; g.rows = rows; g.width = (uint32_t)width; g.vocab = (uint32_t)vocab;
    (void)hipGetLastError();
    of_type(dtype, [&](auto k) { k.loss_rows(g, s); });
    rc = launched("linear cross entropy gradient");
    for (int64_t first = 0; first < vocab && rc == TSGEMM_OK; first += plan.piece) {
        const int64_t columns = vocab - first < plan.piece ? vocab - first : plan.piece;
        const bool last = first + plan.piece >= vocab, several = vocab > plan.piece;
        const uint16_t* const wp = static_cast<const uint16_t*>(weight) + first * ldw;
        LinArgs l = product(plan.logits, rows, columns);
        l.a = g.x; l.lda = ldx; l.b = wp; l.ldb = ldw; l.Ka = l.Kb = (uint32_t)width;
        l.row = g.row; l.dl = dl; l.lddl = plan.ld; l.first = (uint32_t)first;
        of_type(dtype, [&](auto k) { k.product(LIN_KIND_DLOGITS, plan.logits.tile, l, s); });
        rc = launched("linear cross entropy gradient of the logits");
        if (rc == TSGEMM_OK && dx) {
            LinArgs a = product(plan.dx, rows, width);
            a.a = dl; a.lda = plan.ld; a.Ka = (uint32_t)plan.piece;
            a.b = wp; a.ldb = ldw; a.Kb = (uint32_t)columns;
            a.out = out_dx; a.ldo = lddx; a.out_rows = (uint32_t)rows; a.unscale = g.unscale;
            if (plan.dx.splits > 1 || several) a.sums = reinterpret_cast<float*>(w + plan.dx_sums);
            a.add = first > 0;
            of_type(dtype, [&](auto k) {
                k.product(LIN_KIND_DX, plan.dx.tile, a, s);
                if (a.sums && last) k.sum(sum_of(a, a.sums), s);
            });
            rc = launched("linear cross entropy gradient of x");
        }
        if (rc == TSGEMM_OK && dweight) {
            LinArgs a = product(plan.dw, plan.piece, width);
            a.a = dl; a.lda = plan.ld; a.b = g.counted_x; a.ldb = plan.ldx; a.Ka = a.Kb = (uint32_t)rows;
            a.out = out_dw + first * lddw; a.ldo = lddw; a.out_rows = (uint32_t)columns; a.unscale = g.unscale;
            if (plan.dw.splits > 1) a.sums = reinterpret_cast<float*>(w + plan.dw_sums);
            of_type(dtype, [&](auto k) {
                k.product(LIN_KIND_DW, plan.dw.tile, a, s);
                if (a.sums) k.sum(sum_of(a, a.sums), s);
            });
            rc = launched("linear cross entropy gradient of the weight");
        }
    }
    return rc;
}

}  // extern "C"
