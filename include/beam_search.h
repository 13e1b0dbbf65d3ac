/*
 * beam_search.h -- C ABI of a beam search's step on MI355X (gfx950): the best continuations of each
 * request's beams by their logits, and the reordering of the states that follow them.
 *
 * Conventions and the order of validation are gemm_i8.h's. Rows may start at any address aligned to
 * the element.
 */
#ifndef BEAM_SEARCH_H
#define BEAM_SEARCH_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm_dtype.h"
#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most beams of a request, and most continuations beam_step returns for one. */
#define BEAM_MAX 64

/*
 * B requests of W beams each; beam w of request b has row b W + w of the logits (V a row, leading
 * dimension ld) and scores[b W + w], the logarithm of its probability so far. With
 *     lse   = log sum_v exp x_v                     of the beam's row
 *     total = scores + x_v - lse
 * the `top` continuations (beam, token v) of largest total of each request are written, in descending
 * order: out_scores, out_beams (0 to W - 1) and out_tokens, B x top each, packed.
 *   - Totals are compared in 64 bits (lse is a sum in FP32 of terms in FP32); of equal ones the
 *     lower beam comes first, of one beam's equal logits the lower token.
 *   - finished (NULL: none is) holds B W bytes: a beam whose byte is not 0 offers itself alone, with
 *     token pad_token and its score as the total. Its row is not read.
 *   - A continuation of total -infinity or NaN does not count: banned tokens, beams of score
 *     -infinity (those of a first step), rows that hold a NaN or +infinity or nothing but -infinity.
 *     Where fewer than `top` are left, the last entries are score -infinity, beam -1 and token -1.
 *
 * W and top are 1 to BEAM_MAX (else SGEMM_EINVAL_ARG), V at least 1 (else SGEMM_EINVAL_DIM; all where
 * B is at least 1). workspace: beam_step_workspace_size bytes of caller-owned device memory, 16-byte
 * aligned; SGEMM_EINVAL_ARG if smaller. No initialisation needed; calls that share one must not
 * overlap in time. Repeated calls with the same arguments give identical bits.
 */
int beam_step(int B, int W, int V,
              const void *logits, int dtype, int64_t ld,
              const float *scores, const uint8_t *finished, int64_t pad_token,
              int top, float *out_scores, int64_t *out_beams, int64_t *out_tokens,
              void *workspace, size_t workspace_bytes,
              void *stream);

/* Bytes of workspace beam_step needs for this shape on the current device (0 for arguments it would
 * refuse and where no device answers). */
size_t beam_step_workspace_size(int B, int W, int V, int dtype, int top);

/*
 * One tensor of states with a row for each beam, in bytes: row r's piece (i, j), i < count1 and
 * j < count2, is `run` bytes from src + r src_row + i src_step1 + j src_step2, and goes to the same
 * place of dst by its own strides.
 */
typedef struct {
    const void *src;
    void *dst;
    int64_t src_row, dst_row;
    int64_t count1, src_step1, dst_step1;
    int64_t count2, src_step2, dst_step2;
    int64_t run;
} beam_state;

/*
 * Row b W + w of each state's dst gets row b W + beams[b W + w] of its src: the states of the
 * beams that beam_step chose. beams: B W indices of beam_bytes (4 or 8) each; one outside 0 to W - 1
 * (beam_step's -1) stands for w itself. W is 1 to BEAM_MAX.
 *
 * In place where a state's dst is its src, with the same strides; rows that stay are not touched then.
 * Any other overlap of what is written with anything else is SGEMM_EALIAS. States that share an
 * allocation must not interleave their rows, except as disjoint slices of common rows, or, where both
 * are reordered in place, of common pieces (keys and values side by side in each position). Strides and
 * counts are not negative (else SGEMM_EINVAL_DIM), pieces of a dst do not overlap (SGEMM_EINVAL_LD),
 * a state has fewer than 2^35 bytes to a row (SGEMM_ETOO_LARGE). `states` is host memory, read
 * before the call returns.
 */
int reorder_beams(int B, int W, const void *beams, int beam_bytes,
                  const beam_state *states, int count,
                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_SEARCH_H */
