// How blocks of one launch that wait for one another count their arrivals: the rules alone,
// for the kernels and for the host.
#pragma once

#ifdef __CUDACC__
#define MOE_MEET __host__ __device__ constexpr
#else
#define MOE_MEET constexpr
#endif

namespace moe {

// Meetings 0, 1, 2, ...  A block arrives at each of them once, in order, and waits for each in
// order; it may have arrived at the next one before it waits for one, never at the one after that.
// Arrivals are counted in two words in turn: who arrives at meeting k + 2 has waited for meeting k,
// so that a word holds no arrival of meeting k + 2 before all of meeting k.  (In one word for all of
// them a block that is one ahead would stand for one that has not come.)
constexpr int kMeetWords = 2;
MOE_MEET int meet_word(int number) { return number % kMeetWords; }
// what the word holds, at least, once all have arrived at this meeting
MOE_MEET int meet_count(int number, int blocks) { return (number / kMeetWords + 1) * blocks; }

// A block whose wait takes too long marks the word, by compare-and-swap of what it has read there while
// that was too little: then nobody has passed this meeting, and nobody does.  Where no block comes
// ahead, a meeting so ends in the same way for all of them.  (Ahead, a block that still waits for meeting
// k may find the mark of meeting k + 2, and gives up before the others.)
constexpr int kMeetGaveUp = 1 << 30;           // above every count
enum MeetState { kMeetWait, kMeetMet, kMeetEnded };
MOE_MEET int meet_state(int seen, int number, int blocks) {
  return seen & kMeetGaveUp ? kMeetEnded : seen >= meet_count(number, blocks) ? kMeetMet : kMeetWait;
}

}  // namespace moe
