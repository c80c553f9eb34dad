/*
 * trellis_grouped.h -- operations of libtrellis.so whose rows are grouped by
 * an index per row: tokens sorted by expert and back, the experts' coded
 * products, and low-rank adapters of many requests beside one shared
 * projection. The conventions of trellis.h hold (device pointers owned by the
 * caller, dense row-major arrays, outputs overlapping nothing else, work
 * enqueued on `stream`, nothing enqueued on a negative status), with these
 * additions:
 *   - Arrays of bf16, float32 and int32 need the alignment of their element;
 *     workspaces, codes and codebooks need 16 bytes. Rows whose length is a
 *     multiple of 8 in arrays aligned to 16 bytes are moved 16 bytes at a time.
 *   - Group indexes, offsets and positions are read on the device and never
 *     trusted as addresses: an index outside its range selects no row.
 *   - Every sum runs in float32 in an order that the sizes, the indexes and the
 *     current device's number of compute units fix: repeated calls on a device
 *     give identical bits, devices with other numbers may give others.
 *   - No call reads what an earlier call left in its workspace, and every
 *     call may be captured into a graph and replayed with other indexes of
 *     the same sizes. Calls (and graphs) that share a workspace must not
 *     overlap in time.
 */
#ifndef TRELLIS_GROUPED_H
#define TRELLIS_GROUPED_H

#include "trellis.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of groups (experts, adapters) of one call. */
#define TRELLIS_MAX_GROUPS 1024

/* Largest number of slots (tokens x top_k) or rows of one call. */
#define TRELLIS_MAX_SLOTS (1 << 21)

/*
 * Sort slots by group. ids: int32 [tokens][top_k]; slot i = token * top_k +
 * choice. Slots with 0 <= ids[i] < groups are placed in ascending order of
 * their id, slots of one id in ascending order of i; all other slots are
 * dropped.
 *   offsets  int32 [groups + 1]  first place of each group; the last entry is
 *                                the number of placed slots
 *   order    int32 [slots]       the slot at each place, -1 behind the last
 *   position int32 [slots]       the place of each slot, -1 if dropped
 * 0 <= tokens, 1 <= top_k, 1 <= groups <= TRELLIS_MAX_GROUPS, tokens * top_k
 * <= TRELLIS_MAX_SLOTS. An id may occur more than once in a token. With no
 * tokens only `offsets` is written (zeros). workspace: 16-byte aligned, at
 * least trellis_route_workspace_bytes (0 for few slots: may be null then).
 */
int trellis_route(const int32_t *ids, int32_t tokens, int32_t top_k, int32_t groups,
                  int32_t *offsets, int32_t *order, int32_t *position, void *workspace,
                  size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of trellis_route; (size_t)-1 if the sizes are not supported. */
size_t trellis_route_workspace_bytes(int32_t tokens, int32_t top_k, int32_t groups);

/*
 * Copy every token's row to the places of its slots:
 *   out[position[m][j]][:] = x[m][:]   for every slot with a place.
 * x: bf16 [tokens][width]; position: int32 [tokens][top_k] of trellis_route;
 * out: bf16 [tokens * top_k][width], whose rows behind the last placed slot
 * are left as they were. Gradient: trellis_combine of the gradient of `out`
 * without weights. 1 <= width <= 2^19.
 */
int trellis_dispatch(const uint16_t *x, const int32_t *position, int32_t tokens, int32_t top_k,
                     int32_t width, uint16_t *out, hipStream_t stream);

/*
 * Bring the slots' rows back to their tokens and add them up:
 *   out[m][:] = bf16( sum_j weights[m][j] * y[position[m][j]][:] ),
 * j ascending over the slots with a place; a token without any gets zeros.
 * Rows of dropped slots are not read and their weights do not enter (also
 * where either is not finite). y: bf16 [tokens * top_k][width]; weights:
 * float32 [tokens][top_k], or null for the plain sum; out: bf16
 * [tokens][width].
 */
int trellis_combine(const uint16_t *y, const float *weights, const int32_t *position,
                    int32_t tokens, int32_t top_k, int32_t width, uint16_t *out,
                    hipStream_t stream);

/*
 * Gradient of trellis_combine with weights, from dout: bf16 [tokens][width]:
 *   dy[position[m][j]][:] = bf16( weights[m][j] * dout[m][:] )
 *   dweights[m][j]        = sum_h dout[m][h] * y[position[m][j]][h]
 * for every slot with a place; dweights is 0 for dropped slots, and rows of
 * dy behind the last placed slot are left as they were. dy: bf16
 * [tokens * top_k][width]; dweights: float32 [tokens][top_k].
 */
int trellis_combine_backward(const uint16_t *dout, const uint16_t *y, const float *weights,
                             const int32_t *position, int32_t tokens, int32_t top_k,
                             int32_t width, uint16_t *dy, float *dweights, hipStream_t stream);

/*
 * The experts' products over rows sorted by expert (trellis_dispatch):
 *   y[s] = bf16( W_e x[s] )  for the rows s of [offsets[e], offsets[e + 1]),
 * with W_e decoded as in trellis_prefill (axis 1: y = x W^T, axis 0: y = x W;
 * the product of one axis is the gradient with respect to x of the other's,
 * with the same codes, scales and codebook and in/out exchanged).
 * x: bf16 [rows][in]; offsets: int32 [experts + 1] of trellis_route, on the
 * device; codes: uint32 [experts][...], every expert's in the layout of `g`
 * (g describes one expert); scales: float32 [experts][stored rows]; lut:
 * float32 [4096], shared by the experts; y: bf16 [rows][out], whose rows
 * outside every expert are left as they were. Offsets are clamped to [0, rows];
 * ones that are not ascending leave it open which expert's product a row gets,
 * if any. rows <= TRELLIS_MAX_SLOTS. x, codes, lut and y
 * need 16-byte alignment. workspace: 16-byte aligned, at least
 * trellis_experts_workspace_bytes(g, rows, experts) bytes (0 for few rows per
 * expert: may be null then).
 */
int trellis_experts(const uint16_t *x, int32_t rows, const int32_t *offsets, int32_t experts,
                    const uint32_t *codes, const float *scales, const float *lut,
                    const trellis_geometry *g, uint16_t *y, void *workspace,
                    size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of trellis_experts on the current device (its number of compute
 * units decides which tiles a call takes); (size_t)-1 if the sizes are not supported. */
size_t trellis_experts_workspace_bytes(const trellis_geometry *g, int32_t rows, int32_t experts);

/* Largest rank of an adapter, and number of rows of one adapter call. */
#define TRELLIS_MAX_RANK 128
#define TRELLIS_MAX_ADAPTER_ROWS (1 << 20)

/*
 * Low-rank adapters of one projection in -> out, all of one rank (smaller ones
 * are padded with zero rows). Both factors are stored by rank:
 *   a: bf16 [count][rank][in_features], b: bf16 [count][rank][out_features]
 *   (the transpose of a matrix [out][rank]); scales: float32 [count].
 */
typedef struct trellis_adapter_set {
    const uint16_t *a;
    const uint16_t *b;
    const float *scales;
    int32_t count;         /* 1 .. TRELLIS_MAX_GROUPS */
    int32_t rank;          /* 1 .. TRELLIS_MAX_RANK */
    int32_t in_features;   /* 1 .. 2^19, any */
    int32_t out_features;  /* 1 .. 2^19, any */
} trellis_adapter_set;

/*
 * Every row's own adapter beside a projection that all rows share. With
 * i = ids[m] (int32 [rows]):
 *   u[m] = a[i] x[m],   y[m] = bf16( base[m] + scales[i] * b[i]^T u[m] )
 * and y[m] = base[m], u[m] = 0 for rows whose id is outside [0, count).
 * x: bf16 [rows][in]; base: bf16 [rows][out], the shared projection's output
 * (trellis_prefill or trellis_gemv of x), or null for zeros; y: bf16
 * [rows][out], which may be `base` itself (rows without an adapter are then
 * not touched); u: float32 [rows][rank], kept for the backward pass, or null.
 * u, the products and the sums are float32; beyond few rows u enters the second
 * product as three bf16 parts whose sum it is. Where a value of b that a row
 * meets is infinite, y is the formula's infinity or, where a part of u is 0 (its
 * mantissa is short), NaN. workspace: 16-byte aligned, at least
 * trellis_adapters_workspace_bytes(f, rows, 0) bytes.
 */
int trellis_adapters(const uint16_t *x, const int32_t *ids, int32_t rows,
                     const trellis_adapter_set *f, const uint16_t *base, uint16_t *y, float *u,
                     void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of trellis_adapters from dy: bf16 [rows][out], with x, ids and the
 * forward pass's u:
 *   g[m]  = scales[i] * b[i] dy[m]
 *   dx[m] = bf16( base[m] + a[i]^T g[m] )     (base[m] without an adapter)
 *   da[i] = bf16( sum over the rows m of adapter i of g[m] x[m]^T )
 *   db[i] = bf16( sum over the same rows of scales[i] * u[m] dy[m]^T )
 * base: bf16 [rows][in], the shared projection's own gradient (the product of
 * dy with the same codes on the other axis), or null for zeros; dx may be
 * `base` itself. da and db have the factors' layout and are written whole:
 * zeros for adapters without rows (also for rows = 0). Products and sums are
 * float32; beyond few rows g and u enter the second products as three bf16 parts,
 * and an infinity in a, x or dy gives the formula's infinity or, where it meets a
 * part of 0, NaN.
 * workspace: 16-byte aligned, at least
 * trellis_adapters_workspace_bytes(f, rows, 1) bytes.
 */
int trellis_adapters_backward(const uint16_t *dy, const uint16_t *x, const float *u,
                              const int32_t *ids, int32_t rows, const trellis_adapter_set *f,
                              const uint16_t *base, uint16_t *dx, uint16_t *da, uint16_t *db,
                              void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of trellis_adapters (backward = 0) or of its gradient; only
 * the sizes in f are read. (size_t)-1 if they are not supported. */
size_t trellis_adapters_workspace_bytes(const trellis_adapter_set *f, int32_t rows,
                                        int32_t backward);

#ifdef __cplusplus
}
#endif

#endif /* TRELLIS_GROUPED_H */
