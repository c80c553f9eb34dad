/*
 * trellis_mlp.h -- operations of libtrellis.so around an MLP or a layer of
 * experts: the whole layer for few tokens, SwiGLU over many rows with its
 * gradient, and rows kept in 8 bits for a backward pass. The conventions of
 * trellis_grouped.h hold: device pointers owned by the caller, dense row-major
 * arrays aligned to their elements (16 bytes where a function says so), outputs
 * overlapping nothing else, sums in float32 in an order that the sizes, the ids
 * and the device's compute units fix, nothing kept between calls, every call fit
 * for capture; calls that share a workspace must not overlap in time.
 */
#ifndef TRELLIS_MLP_H
#define TRELLIS_MLP_H

#include "trellis_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of tokens, and of choices per token, of trellis_experts_mlp. */
#define TRELLIS_MAX_MLP_TOKENS 32
#define TRELLIS_MAX_MLP_CHOICES 32

/*
 * Coded matrices of several experts, as for trellis_experts: codes uint32
 * [experts][...], every expert's in the layout of `g` (g describes one expert);
 * scales float32 [experts][stored rows]; lut float32 [4096], shared. codes and
 * lut need 16-byte alignment.
 */
typedef struct trellis_expert_set {
    const uint32_t *codes;
    const float *scales;
    const float *lut;
    trellis_geometry g;
} trellis_expert_set;

/*
 * A whole layer of experts for few tokens, in place of trellis_route,
 * trellis_dispatch, trellis_experts, SwiGLU, trellis_experts and trellis_combine:
 *   h_e[m] = w_e[m] * silu(Wg_e x[m]) * (Wu_e x[m]),  silu(v) = v / (1 + exp(-v))
 *   out[m] = bf16( sum over the experts e that token m chose, ascending, of Wd_e h_e[m] )
 * ids: int32 [tokens][top_k]; token m chose e if ids[m][j] = e for some j, and
 * w_e[m] is the sum of its weights[m][j] (float32 [tokens][top_k]; null: ones)
 * for those j. An id outside [0, experts) chooses none; a token without a choice
 * gets zeros. Values that a token did not choose do not enter, also where they
 * are not finite. h enters the second product as two bf16 parts (16 bits of its
 * mantissa; off by up to 2^-132 where that is more), neither of them zero unless h is.
 * x and out: bf16 [tokens][hidden], 16-byte aligned.
 *   up:   axis 1, in = hidden, out = 2 inter: the gate's rows, then the up's
 *   down: either axis, in = inter, out = hidden (axis 1 needs inter % 256 == 0)
 * 0 <= tokens <= TRELLIS_MAX_MLP_TOKENS, 1 <= top_k <= TRELLIS_MAX_MLP_CHOICES,
 * 1 <= experts <= TRELLIS_MAX_GROUPS; with experts = 1 it is a dense MLP, for which
 * trellis_gate_up_swiglu and the down projection's own call, with h in bf16 between
 * them, mostly take less time (by 7 to 28% for 5120 -> 17408 -> 5120).
 * Codes of experts that nobody chose are not read. workspace: 16-byte aligned, at
 * least trellis_experts_mlp_workspace_bytes bytes.
 */
int trellis_experts_mlp(const uint16_t *x, const int32_t *ids, const float *weights, int32_t tokens,
                        int32_t top_k, int32_t experts, const trellis_expert_set *up,
                        const trellis_expert_set *down, uint16_t *out, void *workspace,
                        size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of trellis_experts_mlp on the current device (its number of
 * compute units decides the split); only the geometries in up and down are read.
 * (size_t)-1 if the sizes are not supported. */
size_t trellis_experts_mlp_workspace_bytes(int32_t tokens, int32_t top_k, int32_t experts,
                                           const trellis_expert_set *up,
                                           const trellis_expert_set *down);

/* Largest number of values of one of the calls below (rows x width, for SwiGLU those
 * of [2 rows][inter], every row rounded up to 32), and of rows that are kept. */
#define TRELLIS_MAX_KEPT_VALUES (1ll << 35)
#define TRELLIS_MAX_KEPT_ROWS (1 << 22)

/*
 * Rows of bf16 held in 8 bits. 32 adjacent values of a row (fewer at its end)
 * share one exponent E, the largest exponent field of their bf16 values:
 *   codes      int8  [rows][width]            q = x 2^(133 - E), rounded half to
 *                                             even and cut off at +-127
 *   exponents  uint8 [rows][ceil(width / 32)] E
 * and the value held is q 2^(E - 133), a bf16 value; it is off by at most half of
 * 2^(E - 133), which is at most 1/128 of the group's largest magnitude. A group
 * with an infinity or NaN has E = 255 and stands for NaN throughout.
 */
typedef struct trellis_kept {
    int8_t *codes;
    uint8_t *exponents;
} trellis_kept;

/* Put rows of bf16 away: x bf16 [rows][width]. 0 <= rows <= TRELLIS_MAX_KEPT_ROWS,
 * 1 <= width <= 2^19. */
int trellis_keep(const uint16_t *x, int32_t rows, int32_t width, const trellis_kept *kept,
                 hipStream_t stream);

/* And back: out bf16 [rows][width]. */
int trellis_restore(const trellis_kept *kept, int32_t rows, int32_t width, uint16_t *out,
                    hipStream_t stream);

/*
 * SwiGLU between an MLP's two products (or the experts' two over sorted rows):
 *   h[m] = bf16( silu(g[m]) * u[m] ),   gu: bf16 [rows][2 inter], g in the first
 * half of a row, u in the second; h: bf16 [rows][inter]. With `kept` gu is also
 * put away as trellis_keep would put [2 rows][inter] (g and u of a row are two rows
 * there). 0 <= rows <= TRELLIS_MAX_SLOTS, 1 <= inter <= 2^18.
 */
int trellis_swiglu(const uint16_t *gu, int32_t rows, int32_t inter, uint16_t *h,
                   const trellis_kept *kept, hipStream_t stream);

/*
 * Its gradient from dh: bf16 [rows][inter], with s = 1 / (1 + exp(-g)):
 *   dg = bf16( dh u s (1 + g (1 - s)) ),  du = bf16( dh g s ),  dgu = [dg, du].
 * Exactly one of gu and kept is given. h: null, or bf16 [rows][inter] that gets
 * trellis_swiglu's result again, from the same values (for the gradient of an
 * adapter beside the second product).
 */
int trellis_swiglu_backward(const uint16_t *dh, const uint16_t *gu, const trellis_kept *kept,
                            int32_t rows, int32_t inter, uint16_t *dgu, uint16_t *h,
                            hipStream_t stream);

/* trellis_adapters_backward with x held in 8 bits ([rows][in_features]); the same
 * workspace. */
int trellis_adapters_backward_kept(const uint16_t *dy, const trellis_kept *x, const float *u,
                                   const int32_t *ids, int32_t rows, const trellis_adapter_set *f,
                                   const uint16_t *base, uint16_t *dx, uint16_t *da, uint16_t *db,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TRELLIS_MLP_H */
